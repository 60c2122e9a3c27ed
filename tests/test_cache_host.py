"""The cache operators' checks on the host: what include/pa_cache.h refuses is
refused before any CUDA call, and the plain forms the GPU tests compare with
are pinned by hand-worked values."""
import ctypes
import math
import os
import re

import pytest
import torch

from paged_attention_gb300 import binding as B
from paged_attention_gb300 import build as build_mod

import cache_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(1 << 20)          # aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load()


def problem(**kw):
    p = B.PaProblem(num_seqs=3, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16,
                    num_pages=50, max_pages_per_seq=10, total_q_tokens=3, max_q_len=1,
                    max_context_len=160, layout=0, kv_dtype=B.PA_MX4, num_ctas=152,
                    sm_scale=0.1)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


# arguments of each entry point after the problem, all well formed
GOOD = {
    "pa_kv_append": [FAKE, FAKE, 256, 256] + [FAKE] * 9 + [None],
    "pa_kv_expand": [FAKE] * 8 + [10, 60] + [FAKE] * 3 + [None],
    "pa_decode_mx4": [FAKE] * 9 + [1 << 40] + [FAKE] * 2 + [None],
    "pa_key_weights": [FAKE] * 9 + [None],
    "pa_kv_evict": [100, 4, 32] + [FAKE] * 6 + [ctypes.c_void_p(2 << 20), 7, FAKE,
                                              FAKE, ctypes.c_void_p(3 << 20), FAKE, None],
}


def call(lib, name, p, args=None):
    return getattr(lib, name)(ctypes.byref(p) if p is not None else None,
                              *(GOOD[name] if args is None else args))


def test_every_declared_entry_point_is_exported(lib):
    with open(os.path.join(ROOT, "include", "pa_cache.h")) as f:
        names = re.findall(r"PA_API\s+[\w\s\*]*?\b(pa_\w+)\s*\(", f.read())
    assert set(names) == set(B.EXPORTED_CACHE)
    for n in names:
        assert hasattr(lib, n)


@pytest.mark.parametrize("name", sorted(GOOD))
def test_problems_that_are_refused(lib, name):
    bad = B.PA_ERR_INVALID_ARG
    assert call(lib, name, None) == bad
    for field, value in (("num_seqs", 0), ("num_kv_heads", 3), ("num_pages", 0), ("layout", 2),
                         ("kv_dtype", 3), ("kv_dtype", -1), ("max_pages_per_seq", 9),
                         ("total_q_tokens", -1), ("max_q_len", -1), ("max_q_len", 161),
                         ("max_context_len", -1), ("window", -1), ("mask_q_tiles", 1),
                         ("sm_scale", float("nan")), ("sm_scale", -1.0), ("num_ctas", -1)):
        assert call(lib, name, problem(**{field: value})) == bad, field
    for field, value in (("head_dim", 96), ("head_dim", 256), ("page_size", 48),
                         ("page_size", 8), ("page_size", 512), ("kv_dtype", B.PA_FP8_E4M3),
                         ("q_dtype", B.PA_FP8_E4M3)):
        p = problem(**{field: value, "max_pages_per_seq": 100})
        assert call(lib, name, p) == B.PA_ERR_UNSUPPORTED, field
    if name != "pa_kv_evict":
        assert call(lib, name, problem(max_q_len=0)) == bad


@pytest.mark.parametrize("name", sorted(GOOD))
def test_pointers_that_are_refused(lib, name):
    """Each pointer in turn NULL (where it must not be) and misaligned."""
    optional = {"pa_kv_append": {11, 12}, "pa_kv_expand": {12}, "pa_decode_mx4": {11},
                "pa_key_weights": {8}, "pa_kv_evict": {14}}[name]
    args = GOOD[name]
    for i, a in enumerate(args[:-1]):          # the last one is the stream
        if not isinstance(a, ctypes.c_void_p):
            continue
        if i not in optional:
            st = call(lib, name, problem(), args[:i] + [None] + args[i + 1:])
            assert st == B.PA_ERR_INVALID_ARG, i
        odd = ctypes.c_void_p(a.value + 2)
        assert call(lib, name, problem(), args[:i] + [odd] + args[i + 1:]) == B.PA_ERR_INVALID_ARG, i


def test_refusals_of_their_own(lib):
    a = GOOD["pa_kv_append"]
    for stride in (255, 248, 260):
        assert call(lib, "pa_kv_append", problem(), a[:2] + [stride] + a[3:]) == 1
        assert call(lib, "pa_kv_append", problem(), a[:3] + [stride] + a[4:]) == 1
    # a bf16 cache needs no scales; only evict and weights and append know it
    for name in ("pa_kv_expand", "pa_decode_mx4"):
        assert call(lib, name, problem(kv_dtype=B.PA_BF16)) == B.PA_ERR_UNSUPPORTED
    e = GOOD["pa_kv_expand"]
    assert call(lib, "pa_kv_expand", problem(), e[:8] + [9] + e[9:]) == 1
    assert call(lib, "pa_kv_expand", problem(), e[:9] + [0] + e[10:]) == 1
    d = GOOD["pa_decode_mx4"]
    n = B.pa_mx4_workspace_size(problem())
    assert n > 0
    assert call(lib, "pa_decode_mx4", problem(), d[:9] + [n - 1] + d[10:]) == B.PA_ERR_WORKSPACE
    assert call(lib, "pa_decode_mx4", problem(max_q_len=9)) == B.PA_ERR_UNSUPPORTED   # 36 rows
    assert B.pa_mx4_workspace_size(problem(max_q_len=9)) == 0
    assert B.pa_mx4_workspace_size(problem(max_q_len=8)) > 0
    assert B.pa_mx4_workspace_size(problem(num_ctas=1025)) == 0
    v = GOOD["pa_kv_evict"]
    for budget, first, recent in ((0, 0, 0), (-1, 0, 0), (10, -1, 0), (10, 0, -1), (10, 6, 5),
                                  (100, 2 ** 31 - 1, 2 ** 31 - 1), (113, 0, 0)):
        assert call(lib, "pa_kv_evict", problem(), [budget, first, recent] + v[3:]) == 1
    same_table = v[:9] + [v[8]] + v[10:]
    assert call(lib, "pa_kv_evict", problem(), same_table) == 1
    for shift in (0, 4, 8, -8):                # overlapping length arrays
        over = v[:13] + [ctypes.c_void_p(v[11].value + shift)] + v[14:]
        assert call(lib, "pa_kv_evict", problem(), over) == 1


def test_no_rows_is_no_work(lib):
    p = problem(total_q_tokens=0, max_q_len=0)
    for name in ("pa_kv_append", "pa_kv_expand", "pa_key_weights"):
        args = [a if isinstance(a, int) else None for a in GOOD[name]]
        assert call(lib, name, p, args) == B.PA_OK


def test_no_rows_is_no_work_in_decode(lib):
    """As above, but the workspace is still looked at."""
    p = problem(total_q_tokens=0, max_q_len=0)
    n = B.pa_mx4_workspace_size(p)
    assert n > 0
    rest = [None, None, None]                      # out, lse, stream
    assert call(lib, "pa_decode_mx4", p, [None] * 8 + [FAKE, n] + rest) == B.PA_OK
    assert call(lib, "pa_decode_mx4", p, [None] * 8 + [FAKE, n - 1] + rest) == B.PA_ERR_WORKSPACE
    assert call(lib, "pa_decode_mx4", p, [None] * 9 + [n] + rest) == B.PA_ERR_INVALID_ARG


def test_attention_entry_points_refuse_a_4_bit_cache(lib):
    p = problem()
    assert B.pa_assign_workspace_size(p, B.PA_MODE_DECODE) == 0
    assert B.pa_assign_workspace_size(p, B.PA_MODE_PREFILL) == 0
    assert B.pa_static_workspace_size(p, 0) == 0


def test_binding_checks_new_rows():
    p = problem()
    ok = torch.zeros((3, 2, 128), dtype=torch.bfloat16)
    assert B._new_rows(ok, p, "k_new") == 256
    wide = torch.zeros((3, 1024), dtype=torch.bfloat16)[:, 256:512].unflatten(1, (2, 128))
    assert B._new_rows(wide, p, "k_new") == 1024
    for t in (ok.float(), ok[:2], ok[:, :1], ok[..., :64], ok.transpose(0, 1),
              torch.zeros((3, 128, 2), dtype=torch.bfloat16).transpose(1, 2)):
        with pytest.raises(ValueError):
            B._new_rows(t, p, "k_new")


def test_binding_refuses_what_the_kernels_would_misread():
    wide = torch.zeros((4, 6), dtype=torch.float32)
    assert B._dense(None) is None and B._dense(wide) == wide.data_ptr()
    assert B._dense(wide[1:3]) == wide[1:3].data_ptr()          # whole rows are dense
    for t in (wide[:, :4], wide.t(), wide[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            B._dense(t)
    assert B._ints(None) is None
    with pytest.raises(ValueError, match="int64"):
        B._ints(torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="on cpu"):
        B._ints(torch.zeros(3, dtype=torch.int32))
    codes, rows = torch.zeros(64, dtype=torch.uint8), torch.zeros(64, dtype=torch.bfloat16)
    mx4, bf16 = problem(), problem(kv_dtype=B.PA_BF16)
    assert B._cache(codes, mx4) == codes.data_ptr() and B._cache(rows, bf16) == rows.data_ptr()
    assert B._cache(None, bf16) is None
    for t, p in ((codes, bf16), (rows, mx4)):
        with pytest.raises(ValueError, match="cache for kv_dtype"):
            B._cache(t, p)


def test_binding_refuses_before_the_library_is_called(monkeypatch):
    """Each entry point, every tensor in turn a slice of a wider one, lengths and
    tables in 64 bits, a cache of the other type: refused with nothing called."""
    calls = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: calls.append(name) or 0

    # (CPU tensors stand for device ones)
    monkeypatch.setattr(B, "_lib", Library())
    monkeypatch.setattr(B, "_stream", lambda s: 0)
    ints = B._ints
    monkeypatch.setattr(B, "_ints", lambda t: B._dense(t) if t is None or t.dtype is torch.int32
                        else ints(t))

    def i32(*shape):
        return torch.zeros(shape, dtype=torch.int32)

    def u8(*shape):
        return torch.zeros(shape, dtype=torch.uint8)

    bf, f32 = (lambda *s: torch.zeros(s, dtype=torch.bfloat16)), (lambda *s: torch.zeros(s))
    p, new, q = problem(), bf(3, 2, 128), bf(3, 8, 128)
    table, lens, err = i32(3, 10), i32(3), i32(1)
    cache, scale, pages = u8(50, 16, 2, 64), u8(50, 16, 2, 4), bf(50, 16, 2, 128)
    lse, w = f32(3, 8), f32(50, 2, 16)
    whole = {
        "pa_kv_append": [p, new, new, table, lens, lens, cache, scale, cache, scale, w, err],
        "pa_kv_expand": [p, cache, scale, cache, scale, table, lens, lens, table, 50, pages, pages,
                         err],
        "pa_decode_mx4": [p, q, cache, scale, cache, scale, table, lens, lens, u8(1 << 20), q, lse],
        "pa_key_weights": [p, q, cache, scale, table, lens, lens, lse, w, err],
        "pa_kv_evict": [p, 9, 1, 2, cache, scale, cache, scale, w, table, table, lens, i32(3, 2, 9),
                        lens, err],
    }
    for name, args in whole.items():
        fn = getattr(B, name)
        fn(*args)
        assert calls == [name]
        for i, a in enumerate(args):
            if not isinstance(a, torch.Tensor) or (name == "pa_kv_append" and i in (1, 2)):
                continue
            if a.numel() > 1:
                wider = torch.zeros(a.shape[:-1] + (a.shape[-1] + 1,), dtype=a.dtype)
                strided = (wider[..., :-1] if a.dim() > 1
                           else torch.zeros(2 * len(a), dtype=a.dtype)[::2])
                with pytest.raises(ValueError):
                    fn(*args[:i], strided, *args[i + 1:])
            if a.dtype is torch.int32:
                with pytest.raises(ValueError):
                    fn(*args[:i], a.long(), *args[i + 1:])
        if name not in ("pa_kv_expand", "pa_decode_mx4"):      # these take 4-bit caches alone
            with pytest.raises(ValueError):
                fn(problem(kv_dtype=B.PA_BF16), *args[1:])
        assert calls == [name]
        calls.clear()


def test_stream_handles(monkeypatch):
    """The current stream's handle, with torch's unnamed call for it and without."""
    class Stream:
        cuda_stream = 77

    monkeypatch.setattr(B.torch.cuda, "current_stream", lambda: Stream())
    monkeypatch.setattr(B, "_raw_stream", None)
    assert B._stream(None) == 77
    monkeypatch.setattr(B, "_raw_stream", lambda dev: 100 + dev)
    assert B._stream(None) == 99                             # -1: the current device
    assert B._stream(Stream()) == 77 and B._stream(5) == 5


def test_plain_quantisation_by_hand():
    x = torch.zeros((1, 64), dtype=torch.float64)
    # largest 6.0: exponent 2 - 2 = 0, scale byte 127; the values are their own codes
    x[0, :8] = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
    x[0, 8:12] = torch.tensor([-0.5, 0.25, 0.75, 5.0])      # ties go to the even code
    # second block: largest 0.4, floor(log2) = -2, scale 2^-4: 6.4 -> 6
    x[0, 32:34] = torch.tensor([0.4, -0.1])
    codes, sc = R.quantise(x)
    assert sc.tolist() == [[127, 123]]
    assert codes[0, :6].tolist() == [0x10, 0x32, 0x54, 0x76, 0x09, 0x62]
    assert codes[0, 16].item() == 0xB7                      # 6 and -1.6 -> -1.5
    back = R.dequantise(codes, sc)
    assert back[0, :8].tolist() == x[0, :8].tolist()
    assert back[0, 32:34].tolist() == [0.375, -0.09375]
    codes, sc = R.quantise(torch.tensor([[math.inf] + [1.0] * 31]))
    assert sc.tolist() == [[255]] and not codes.any()


def test_plain_selection_by_hand():
    w = [0.1, 0.9, 0.5, 0.5, 0.5, math.nan, 0.2, 0.0]
    assert R.select(w, 4, 1, 1) == [0, 1, 2, 7]
    assert R.select(w, 5, 0, 0) == [1, 2, 3, 4, 6]
    assert R.select(w, 7, 0, 0) == [0, 1, 2, 3, 4, 6, 7]
    assert R.select(w, 8, 0, 0) is None
