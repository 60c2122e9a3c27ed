"""The checks on the host of the operators of a serving step: what include/pa_step.h
refuses is refused before any CUDA call; rotary frequencies; and pins of the plain
forms the GPU tests compare with."""
import ctypes
import math
import os
import re
from fractions import Fraction

import pytest
import torch

from paged_attention_gb300 import binding as B
from paged_attention_gb300 import build as build_mod

import step_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def at(n):
    return ctypes.c_void_p(n << 20)      # aligned, never dereferenced


FAKE = at(1)


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load()


def problem(**kw):
    p = B.PaProblem(num_seqs=3, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16,
                    num_pages=50, max_pages_per_seq=10, total_q_tokens=3, max_q_len=1,
                    max_context_len=160, layout=0, kv_dtype=B.PA_BF16, num_ctas=152,
                    sm_scale=0.1)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


ROPE = B.PaRope(rotary_dim=128, interleaved=0, cos_sin_scale=1.0)

# arguments of each entry point after the problem, all well formed
GOOD = {
    "pa_pages_take": [at(1), at(2), at(3), at(4), at(5), at(6), at(7), at(8), at(9), at(10),
                      at(11), None],
    "pa_pages_return": [at(1), at(2), at(3), at(4), at(5), at(6), at(7), None],
    "pa_rope_append": [ctypes.byref(ROPE), at(1), at(2), at(3), at(4), 1024, 256, 256, at(5),
                       at(6), at(7), at(8), at(9), at(10), at(11), at(12), None],
    "pa_page_bounds": [at(1), at(2), at(3), at(4), at(5), None],
    "pa_select_pages": [4, 1, 2] + [at(i) for i in range(1, 9)] + [None],
    "pa_decode_selected": [4] + [at(i) for i in range(1, 9)] + [1 << 40, at(9), at(10), None],
}
# pointers that may be NULL (device_error, lse; a bf16 cache's scales)
OPTIONAL = {"pa_pages_take": {10}, "pa_pages_return": {6}, "pa_rope_append": {12, 14, 15},
            "pa_page_bounds": {4}, "pa_select_pages": {10}, "pa_decode_selected": {11}}


def call(lib, name, p, args=None):
    return getattr(lib, name)(ctypes.byref(p) if p is not None else None,
                              *(GOOD[name] if args is None else args))


def swap(name, i, x):
    a = list(GOOD[name])
    a[i] = x
    return a


def test_every_declared_entry_point_is_exported(lib):
    with open(os.path.join(ROOT, "include", "pa_step.h")) as f:
        text = f.read()
    names = re.findall(r"PA_API\s+[\w\s\*]*?\b(pa_\w+)\s*\(", text)
    assert set(names) == set(B.EXPORTED_STEP)
    for n in names:
        assert hasattr(lib, n)
    assert f"PA_DEV_NO_PAGES = {B.PA_DEV_NO_PAGES}" in text
    for i, n in enumerate(("NONE", "LINEAR", "NTK", "YARN", "BANDS")):
        assert f"PA_ROPE_{n} = {i}" in text and getattr(B, "PA_ROPE_" + n) == i


@pytest.mark.parametrize("name", sorted(GOOD))
def test_problems_that_are_refused(lib, name):
    assert call(lib, name, None) == B.PA_ERR_INVALID_ARG
    for field, value in (("num_seqs", 0), ("num_kv_heads", 3), ("num_pages", 0), ("layout", 2),
                         ("kv_dtype", 3), ("kv_dtype", -1), ("max_pages_per_seq", 9),
                         ("total_q_tokens", -1), ("max_q_len", -1), ("max_q_len", 161),
                         ("max_context_len", -1), ("window", -1), ("mask_q_tiles", 1),
                         ("sm_scale", float("nan")), ("sm_scale", -1.0), ("num_ctas", -1)):
        assert call(lib, name, problem(**{field: value})) == B.PA_ERR_INVALID_ARG, field
    for field, value in (("head_dim", 96), ("head_dim", 256), ("page_size", 48),
                         ("page_size", 8), ("page_size", 512)):
        p = problem(**{field: value, "max_pages_per_seq": 100})
        assert call(lib, name, p) == B.PA_ERR_UNSUPPORTED, field
    if name in ("pa_rope_append", "pa_page_bounds", "pa_decode_selected"):
        for field in ("kv_dtype", "q_dtype"):
            p = problem(**{field: B.PA_FP8_E4M3})
            assert call(lib, name, p) == B.PA_ERR_UNSUPPORTED, field
    if name in ("pa_page_bounds", "pa_decode_selected"):
        assert call(lib, name, problem(kv_dtype=B.PA_MX4)) == B.PA_ERR_UNSUPPORTED
    if name in ("pa_pages_take", "pa_rope_append", "pa_page_bounds"):
        assert call(lib, name, problem(num_pages=1 << 27)) == B.PA_ERR_UNSUPPORTED   # 2^31 slots


@pytest.mark.parametrize("name", sorted(GOOD))
def test_pointers_that_are_refused(lib, name):
    """Each pointer in turn NULL (where it must not be) and misaligned."""
    args = GOOD[name]
    for i, a in enumerate(args[:-1]):          # the last one is the stream
        if not isinstance(a, ctypes.c_void_p):
            continue
        if i not in OPTIONAL[name]:
            assert call(lib, name, problem(), swap(name, i, None)) == B.PA_ERR_INVALID_ARG, i
        if name == "pa_rope_append" and i in (12, 14):
            continue                           # (a bf16 cache's scales are not looked at)
        odd = ctypes.c_void_p(a.value + 2)
        assert call(lib, name, problem(), swap(name, i, odd)) == B.PA_ERR_INVALID_ARG, i


def test_refusals_of_their_own(lib):
    bad, no = B.PA_ERR_INVALID_ARG, B.PA_ERR_UNSUPPORTED
    # outputs that every CTA would read as inputs
    t = GOOD["pa_pages_take"]
    for i, j in ((5, 0), (5, 1), (5, 4), (9, 4), (9, 0), (9, 1), (9, 5)):
        assert call(lib, "pa_pages_take", problem(), swap("pa_pages_take", i, t[j])) == bad
    for j in (0, 1):                          # the last of three lengths
        last = ctypes.c_void_p(t[j].value + 8)
        assert call(lib, "pa_pages_take", problem(), swap("pa_pages_take", 9, last)) == bad
    assert call(lib, "pa_pages_return", problem(),
                swap("pa_pages_return", 5, GOOD["pa_pages_return"][4])) == bad
    r = "pa_rope_append"
    for dim, inter, scale in ((0, 0, 1.0), (8, 0, 1.0), (24, 0, 1.0), (144, 0, 1.0), (-16, 0, 1.0),
                              (128, 2, 1.0), (128, -1, 1.0), (128, 0, math.inf),
                              (128, 0, math.nan)):
        x = B.PaRope(rotary_dim=dim, interleaved=inter, cos_sin_scale=scale)
        assert call(lib, r, problem(), swap(r, 0, ctypes.byref(x))) == bad, (dim, inter, scale)
    assert call(lib, r, problem(head_dim=64)) == bad                 # 128 of 64 elements
    assert call(lib, r, problem(), swap(r, 0, None)) == bad
    for i, least in ((5, 1024), (6, 256), (7, 256)):
        for stride in (least - 1, least - 8, least + 4):
            assert call(lib, r, problem(), swap(r, i, stride)) == bad
    assert call(lib, r, problem(), swap(r, 2, None)) == bad          # q_out without q
    assert call(lib, r, problem(kv_dtype=B.PA_MX4), swap(r, 12, None)) == bad
    s = "pa_select_pages"
    for budget, first, recent in ((0, 0, 0), (-1, 0, 0), (4, -1, 0), (4, 0, -1), (4, 3, 2),
                                  (4, 2 ** 31 - 1, 2 ** 31 - 1)):
        assert call(lib, s, problem(), [budget, first, recent] + GOOD[s][3:]) == bad
    assert call(lib, s, problem(num_q_heads=130)) == no              # 65 heads a KV head
    far = dict(max_pages_per_seq=1 << 20, max_context_len=16 * 45056 + 1)
    assert call(lib, s, problem(**far)) == no
    d = "pa_decode_selected"
    n = B.pa_selected_workspace_size(problem(), 4)
    assert n > 0
    i = 9
    assert call(lib, d, problem(), swap(d, i, n - 1)) == B.PA_ERR_WORKSPACE
    assert call(lib, d, problem(), [0] + GOOD[d][1:]) == bad
    for kw in (dict(num_q_heads=66), dict(num_q_heads=130, head_dim=64), dict(num_ctas=1025)):
        assert call(lib, d, problem(**kw)) == no
        assert B.pa_selected_workspace_size(problem(**kw), 4) == 0
    assert B.pa_selected_workspace_size(problem(num_q_heads=64), 4) > 0
    assert B.pa_selected_workspace_size(problem(num_q_heads=128, head_dim=64), 4) > 0
    assert B.pa_selected_workspace_size(problem(), 0) == 0


@pytest.mark.parametrize("name", ["pa_rope_append", "pa_page_bounds", "pa_select_pages",
                                  "pa_decode_selected"])
def test_no_rows_is_nothing_to_do(lib, name):
    args = [None if isinstance(a, ctypes.c_void_p) else a for a in GOOD[name]]
    if name == "pa_decode_selected":
        args[8] = at(9)                       # its workspace is checked all the same
    assert call(lib, name, problem(total_q_tokens=0, max_q_len=0), args) == B.PA_OK


def test_the_binding_refuses_what_would_be_misread():
    p = problem()
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError):           # lengths on the host
        B.pa_pages_take(p, i32(3), i32(3), i32(3, 10), i32(50), i32(1), i32(3), i32(3), i32(3),
                        i32(3), i32(1))
    k = bf(50, 16, 2, 128)
    rows = (bf(3, 8, 128), bf(3, 2, 128), bf(3, 2, 128))
    steps = torch.zeros(64, dtype=torch.int64)
    for bad in ((rows[0][:2], rows[1], rows[2]), (rows[0], rows[1].float(), rows[2]),
                (rows[0], rows[1], bf(3, 2, 256)[..., ::2]), (bf(3, 128, 8).mT, rows[1], rows[2])):
        with pytest.raises(ValueError):
            B.pa_rope_append(p, ROPE, steps, *bad, i32(3), i32(3), bf(3, 8, 128), k, None, k, None)
    with pytest.raises(ValueError):
        B.pa_rope_append(p, ROPE, steps[:63], *rows, i32(3), i32(3), bf(3, 8, 128), k, None, k,
                         None)
    for f in (lambda: B._typed(bf(4, 4).t(), torch.bfloat16), lambda: B._typed(bf(4), torch.int8),
              lambda: B._here(bf(4)),
              lambda: B._i32(torch.zeros(4, dtype=torch.int64)),
              lambda: B._i32(i32(4, 2)[:, 0])):
        with pytest.raises(ValueError):
            f()


@pytest.mark.parametrize("name", ["pa_pages_take", "pa_rope_append", "pa_page_bounds",
                                  "pa_select_pages", "pa_decode_selected"])
def test_more_rows_than_are_counted_are_refused(lib, name):
    assert call(lib, name, problem(total_q_tokens=(1 << 30) + 1)) == B.PA_ERR_UNSUPPORTED


def test_unit_costs_that_cannot_be_counted_are_refused(lib):
    """A kernel would count a unit's tiles and its cost in 32 bits, and all units' times the
    CTAs in 64."""
    d, most = "pa_decode_selected", 2 ** 31 - 1
    size = lambda budget=4, **kw: B.pa_selected_workspace_size(problem(**kw), budget)  # noqa: E731
    # a list of 4 pages of 16 is one tile, of 10 pages three; rows together list twice as many
    for kw, budget, tiles in ((dict(), 4, 1), (dict(), 10, 3), (dict(), 1 << 20, 3),
                              (dict(max_q_len=2), 4, 2)):
        assert size(budget, unit_cost=most - tiles, **kw) > 0
        for cost in (most - tiles + 1, most):
            assert size(budget, unit_cost=cost, **kw) == 0
            args = [budget] + GOOD[d][1:]
            assert call(lib, d, problem(unit_cost=cost, **kw), args) == B.PA_ERR_UNSUPPORTED
    rows = 1 << 27                            # 2^28 rows and heads
    assert size(total_q_tokens=rows, unit_cost=(1 << 24) - 1) > 0
    assert size(total_q_tokens=rows, unit_cost=1 << 24) == 0
    assert call(lib, d, problem(total_q_tokens=rows, unit_cost=1 << 24)) == B.PA_ERR_UNSUPPORTED
    assert size(unit_cost=-2 ** 31) > 0       # none


def test_lists_that_no_size_holds_are_refused(lib):
    """2^30 + 2 rows and heads of 2^31 - 1 entries of 8 bytes: 2^35 bytes past 2^64."""
    d, budget = "pa_decode_selected", 2 ** 31 - 1
    kw = dict(total_q_tokens=(1 << 29) + 1, max_q_len=2)
    assert B.pa_selected_workspace_size(problem(**kw), budget) == 0
    assert call(lib, d, problem(**kw), [budget] + GOOD[d][1:]) == B.PA_ERR_UNSUPPORTED
    most = (1 << 56) // ((1 << 30) + 2)
    assert B.pa_selected_workspace_size(problem(**kw), most) > 8 * most * (1 << 30)
    assert B.pa_selected_workspace_size(problem(**kw), most + 1) == 0


@pytest.mark.parametrize("name,outputs,sizes", [
    # 3 sequences, 3 rows, 50 pages, a table of 3 x 10; in the arguments' order
    ("pa_pages_take", {2, 5, 6, 7, 8, 9}, [12, 12, 120, 200, 4, 12, 12, 12, 12, 4]),
    ("pa_pages_return", {3, 5}, [12, 12, 120, 200, 4, 4]),
])
def test_outputs_of_the_page_operators_stay_off_everything_else(lib, name, outputs, sizes):
    """Each output on the first and on the last word of every other argument."""
    for i in outputs:
        for j in set(range(len(sizes))) - {i}:
            first = GOOD[name][j].value
            for at_byte in (first, first + sizes[j] - 4, first - sizes[i] + 4):
                args = swap(name, i, ctypes.c_void_p(at_byte))
                assert call(lib, name, problem(), args) == B.PA_ERR_INVALID_ARG, (i, j, at_byte)


def test_queries_in_place_are_dense(lib):
    r = "pa_rope_append"
    for stride in (1032, 1536):
        args = swap(r, 5, stride)
        args[10] = args[2]
        assert call(lib, r, problem(), args) == B.PA_ERR_INVALID_ARG


def test_queries_are_written_where_nothing_is_read(lib):
    """q_out a little before or behind q, or on new keys or values."""
    r, out, word = "pa_rope_append", 10, 16
    args = GOOD[r]
    bad = [args[2].value + word, args[2].value - word,                   # q, all but in place
           args[2].value + 3 * 2048 - word, args[2].value - 3 * 2048 + word]
    for i in (3, 4):                          # k_new, v_new: 3 tokens of 512 bytes
        bad += [args[i].value, args[i].value + 3 * 512 - word, args[i].value - 3 * 2048 + word]
    for x in bad:
        assert call(lib, r, problem(), swap(r, out, ctypes.c_void_p(x))) == B.PA_ERR_INVALID_ARG
    # strided tokens: up to the last one's end
    args = swap(r, 5, 4096)
    args[out] = ctypes.c_void_p(args[2].value + 2 * 8192 + 2048 - word)
    assert call(lib, r, problem(), args) == B.PA_ERR_INVALID_ARG
    # a fused projection's only token turned in place is beside its keys, not on them
    args = swap(r, out, args[2])
    args[3] = ctypes.c_void_p(args[2].value + 2048 - word)
    assert call(lib, r, problem(total_q_tokens=1), args) == B.PA_ERR_INVALID_ARG


# ------------------------------------------------------------- frequencies

def scaling(kind, dim, **kw):
    x = dict(base=10000.0, factor=4.0, original_context=4096.0, high_turns=32.0, low_turns=1.0)
    x.update(kw)
    return B.PaRopeScaling(kind=kind, rotary_dim=dim, **x)


def test_frequencies(lib):
    plain, one = B.pa_rope_inv_freq(scaling(B.PA_ROPE_NONE, 64))
    want = torch.tensor([10000.0 ** (-2 * i / 64) for i in range(32)], dtype=torch.float64)
    assert one == 1.0 and torch.allclose(plain, want, rtol=1e-14, atol=0)
    line, one = B.pa_rope_inv_freq(scaling(B.PA_ROPE_LINEAR, 64))
    assert one == 1.0 and torch.allclose(line, want / 4, rtol=1e-14, atol=0)
    ntk, _ = B.pa_rope_inv_freq(scaling(B.PA_ROPE_NTK, 64))
    base = 10000.0 * 4.0 ** (64 / 62)
    assert torch.allclose(ntk, torch.tensor([base ** (-2 * i / 64) for i in range(32)],
                                            dtype=torch.float64), rtol=1e-13, atol=0)
    # the base was chosen so that the slowest pair is divided by the factor as a whole
    assert math.isclose(float(ntk[-1]), float(want[-1]) / 4, rel_tol=1e-12)
    for kind in (B.PA_ROPE_YARN, B.PA_ROPE_BANDS):
        f, factor = B.pa_rope_inv_freq(scaling(kind, 64))
        assert math.isclose(factor, 0.1 * math.log(4.0) + 1 if kind == B.PA_ROPE_YARN else 1.0)
        turns = 4096.0 * want / (2 * math.pi)
        ratio = f / want
        assert torch.all((ratio >= 0.25 - 1e-12) & (ratio <= 1 + 1e-12))
        assert torch.all(ratio[:-1] >= ratio[1:] - 1e-12)      # faster pairs keep more
        assert float(ratio[0]) == 1.0 and math.isclose(float(ratio[-1]), 0.25)
        if kind == B.PA_ROPE_BANDS:
            assert torch.all(ratio[turns >= 32] == 1)
            assert torch.allclose(ratio[turns <= 1], torch.tensor(0.25, dtype=torch.float64))
            mid = (turns > 1) & (turns < 32)
            kept = (turns[mid] - 1) / 31
            assert torch.allclose(ratio[mid], 0.25 * (1 - kept) + kept, rtol=1e-12)
        else:
            # ends at whole pair indices around those of 32 turns and of one
            at_turns = lambda t: 64 * math.log(4096.0 / (t * 2 * math.pi)) / (2 * math.log(1e4))  # noqa: E731,E501
            lo, hi = math.floor(at_turns(32)), math.ceil(at_turns(1))
            for i in range(32):
                r = min(1.0, max(0.0, (i - lo) / (hi - lo)))
                assert math.isclose(float(ratio[i]), 1 - r + r / 4, rel_tol=1e-12)


@pytest.mark.parametrize("dim", [2, 16, 64, 128])
def test_frequencies_at_the_ends_of_what_is_accepted(lib, dim):
    """Pairs above high_turns as they are, below low_turns divided, whatever the parameters: all
    of them above, all below, all between, and each kind of mixture."""
    kinds = set()
    for base in (1.001, 4.0, 10.0, 1e4, 1e6, 1e30):
        for context in (1.0, 4.0, 6.3, 32.0, 300.0, 4096.0, 1e5, 1e9, 1e300):
            for high, low in ((32.0, 1.0), (32.0, 8.0), (1.5, 1.0), (1e6, 1e-6)):
                for kind in (B.PA_ROPE_YARN, B.PA_ROPE_BANDS):
                    f, _ = B.pa_rope_inv_freq(scaling(kind, dim, base=base, high_turns=high,
                                                      original_context=context, low_turns=low))
                    plain = [base ** (-2 * i / dim) for i in range(dim // 2)]
                    of = []
                    for i, (x, y) in enumerate(zip(f.tolist(), plain)):
                        turns = context * y / (2 * math.pi)
                        # (indices and turns are taken by logarithms: near an end either is right)
                        if turns > high * (1 + 1e-9):
                            assert math.isclose(x, y, rel_tol=1e-12), (base, context, high, low, i)
                            of.append("above")
                        elif turns < low * (1 - 1e-9):
                            assert math.isclose(x, y / 4, rel_tol=1e-12), (base, context, high, low, i)
                            of.append("below")
                        else:
                            assert y / 4 * (1 - 1e-12) <= x <= y * (1 + 1e-12)
                            of.append("between")
                    kinds.add(tuple(sorted(set(of))))
    assert {("above",), ("below",), ("between",)} <= kinds
    if dim > 2:
        assert ("above", "below", "between") in kinds


@pytest.mark.parametrize("dim", [16, 32, 64, 128])
def test_yarn_frequencies_are_the_published_ones(lib, dim):
    """Where the published ends do not meet: its line between them, cut to [0, dim - 1]."""
    for base in (1e4, 1.5e5, 5e5, 1e6):
        for context in (300.0, 2048.0, 4096.0, 8192.0, 32768.0, 262144.0, 1e6):
            for high, low in ((32.0, 1.0), (64.0, 1.0), (32.0, 2.0)):
                at = lambda t: dim * math.log(context / (t * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731,E501
                lo, hi = max(0.0, math.floor(at(high))), min(dim - 1.0, math.ceil(at(low)))
                assert 0 <= lo < hi
                f, _ = B.pa_rope_inv_freq(scaling(B.PA_ROPE_YARN, dim, base=base, high_turns=high,
                                                  original_context=context, low_turns=low))
                for i, x in enumerate(f.tolist()):
                    r = min(1.0, max(0.0, (i - lo) / (hi - lo)))
                    y = base ** (-2 * i / dim)
                    assert math.isclose(x, y / 4 * r + y * (1 - r), rel_tol=1e-13)


def test_frequencies_that_are_refused(lib):
    for kind, dim, kw in ((5, 64, {}), (-1, 64, {}), (0, 0, {}), (0, 63, {}), (0, 130, {}),
                          (0, 64, dict(base=1.0)), (0, 64, dict(base=math.nan)),
                          (1, 64, dict(factor=0.5)), (1, 64, dict(factor=math.inf)), (2, 2, {}),
                          (3, 64, dict(low_turns=0.0)), (4, 64, dict(high_turns=1.0)),
                          (3, 64, dict(original_context=0.0))):
        with pytest.raises(B.PaError):
            B.pa_rope_inv_freq(scaling(kind, dim, **kw))
    for bad in ([math.nan], [math.inf], []):
        with pytest.raises(B.PaError):
            B.pa_rope_steps(bad)


def test_steps_are_turns(lib):
    # 2 pi to 40 digits
    two_pi = Fraction("6.283185307179586476925286766559005768394")
    freq = [1.0, 0.5, 1e-7, 0.0, 2 * math.pi, 10.0, -1.0, 3.0e-39]
    steps = [int(x) & (2 ** 64 - 1) for x in B.pa_rope_steps(freq)]
    for f, s in zip(freq, steps):
        turns = Fraction(f) / two_pi
        far = (Fraction(s, 2 ** 64) - turns) % 1
        far = min(far, 1 - far)
        # a quotient in 53 bits, its divisor rounded: two half steps of 2^-53 of the turns,
        # the fraction below one turn rounded once more, and the last of 64 bits
        assert far <= abs(turns) * Fraction(2, 2 ** 53) + Fraction(1, 2 ** 53) + Fraction(1, 2 ** 64)
    assert steps[3] == 0
    # at a position of a million the angle is still good to 32 bits
    pos, i = 1000003, 0
    far = (Fraction(pos * steps[i], 2 ** 64) - pos * Fraction(freq[i]) / two_pi) % 1
    assert min(far, 1 - far) < Fraction(1, 2 ** 32)


# ------------------------------------------------ pins of the plain forms

def test_plain_pages():
    table = [[7, 3, -1], [5, -1, -1], [-1, -1, -1]]
    got = R.take([5, 4, 0], [3, 1, 6], table, [0, 1, 2, 4, 6], 5, page=4, pages=8, rows=12,
                 max_q=6, max_ctx=12)
    assert got == ([[7, 3, -1], [5, 6, -1], [4, 2, -1]], [8, 5, 6],
                   [(0, 5, 13), (0, 6, 14), (0, 7, 15), (1, 4, 24)]
                   + [(2, 0, 16), (2, 1, 17), (2, 2, 18), (2, 3, 19), (2, 4, 8), (2, 5, 9)]
                   + [R.PAD] * 2, 2, 0)
    stack, count, err = R.give_back([8, 5, 6], [8, 0, 3], got[0], [0, 1, -1, -1, -1], 2, page=4,
                                    pages=5, max_ctx=12)
    assert (stack, count, err) == ([0, 1, -1, -1, 2], 5, 2)   # 5 and 6 are none of 5 pages


def test_plain_bounds_and_selection():
    k = torch.tensor([[1.0, -2.0, 0.0, 127.0], [3.0, -1.0, 0.0, -1.0]])
    b, s = R.bounds(k)
    assert s == 1.0 and b.tolist() == [[3, -1, 0, 127], [1, -2, 0, -1]]
    b, s = R.bounds(k + torch.tensor([0.0, 0.0, 0.0, 1.0]))
    assert s == 2.0 and b.tolist() == [[2, 0, 0, 64], [0, -1, 0, 0]]
    assert R.exponent(0.0) == -50 and R.exponent(127.0) == 0 and R.exponent(127.5) == 1
    assert R.exponent(1e30) == 50 and R.exponent(math.inf) == 50 and R.exponent(0.99) == -7
    bnd = torch.zeros((4, 2, 4))
    bnd[:, 0], bnd[:, 1] = torch.tensor([1.0, 3.0, 2.0, 3.0])[:, None], -1.0
    q = torch.tensor([[1.0, 0.0, 0.0, 0.0]])
    kw = dict(budget=2, num_first=0, num_recent=1, page=16, pages=4, window=0)
    assert R.select(q, bnd, torch.ones(4), [0, 1, 2, 3, 0], 70, **kw) == [1, 4]
    assert R.select(-q, bnd, torch.ones(4), [0, 1, 2, 3, 0], 70, **kw) == [0, 4]   # a tie
    assert R.select(q, bnd, torch.ones(4), [0, 1, 2, 3, 0], 20, **kw) == [0, 1]
    assert R.select(q, bnd, torch.ones(4), [0, 1, 2, 3, 0], 70, **dict(kw, window=7)) == [4, -1]
