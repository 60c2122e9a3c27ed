"""The operators of a serving step (include/pa_step.h) against their 64-bit plain
forms, and together as a decode loop uses them."""
import math

import pytest
import torch

from paged_attention_gb300 import binding as B

import cache_ref as C
import step_ref as R

pytestmark = pytest.mark.gpu

BF16, HALF = torch.bfloat16, 2.0 ** -8        # a rounding to bf16 is off by half a step at most


def ints(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def problem(**kw):
    d = dict(num_seqs=1, num_q_heads=4, num_kv_heads=2, head_dim=128, page_size=16, num_pages=8,
             max_pages_per_seq=8, total_q_tokens=1, max_q_len=1, max_context_len=128, layout=0,
             kv_dtype=B.PA_BF16, sm_scale=0.1)
    d.update(kw)
    return B.PaProblem(**d)


def no_error(err):
    assert int(err) == 0


# ------------------------------------------------------------------- pages

def run_take(seq, q, table, stack, count, *, page, pages, rows, max_q, max_ctx, kv=B.PA_BF16):
    width = len(table[0])
    p = problem(num_seqs=len(seq), page_size=page, num_pages=pages, max_pages_per_seq=width,
                total_q_tokens=rows, max_q_len=max_q, max_context_len=max_ctx, kv_dtype=kv)
    t, err = ints(table), ints([0])
    ctx, left = ints([-9] * len(seq)), ints([-9])
    maps = [ints([-9] * rows) for _ in range(3)]
    stack = ints(stack)
    before = stack.clone()
    B.pa_pages_take(p, ints(seq), ints(q), t, stack, ints([count]), ctx, *maps, left, err)
    torch.cuda.synchronize()
    assert torch.equal(stack, before)
    return (t.tolist(), ctx.tolist(), list(zip(*(m.tolist() for m in maps))), int(left), int(err))


def take_case(seq, q, *, page=16, spare=3, short=0, pad=0, seed=0, holes=()):
    g = torch.Generator().manual_seed(seed)
    have = [R.up(n, page) for n in seq]
    need = [R.up(n + x, page) - h for n, x, h in zip(seq, q, have)]
    pages = sum(have) + sum(need) + spare
    perm = torch.randperm(pages, generator=g).tolist()
    width = max(1, max(h + n for h, n in zip(have, need)))
    table, at = [], 0
    for h in have:
        table.append(perm[at:at + h] + [-1] * (width - h))
        at += h
    for b, j in holes:
        table[b][j] = pages + 5
    stack = perm[at:] + [-1] * at
    return dict(table=table, stack=stack, count=len(perm) - at - short), dict(
        page=page, pages=pages, rows=sum(q) + pad, max_q=max(q), max_ctx=width * page)


@pytest.mark.parametrize("seq,q,kw", [
    ([0], [1], {}), ([15], [1], {}), ([16], [1], {}), ([17], [40], {}), ([5, 0, 31], [1, 1, 1], {}),
    ([5, 0, 31, 16], [0, 33, 0, 16], dict(page=32)), ([0, 0, 0], [0, 0, 5], {}),
    ([100, 1, 64, 255], [3, 70, 2, 1], dict(page=64, pad=7)), ([7] * 3, [300, 1, 129], dict(page=256)),
    ([5, 20, 0, 40], [30, 1, 50, 9], dict(spare=0)), ([5, 20, 0, 40], [30, 1, 50, 9], dict(spare=0, short=1)),
    ([5, 20, 0, 40], [30, 1, 50, 9], dict(spare=0, short=5)),
    ([5, 20, 16, 40], [30, 1, 50, 9], dict(holes=[(0, 0), (2, 0)])),
    (list(range(1300)), [1] * 1300, dict(pad=11)),             # more sequences than a round
    ([3 * i % 50 for i in range(700)], [i % 5 for i in range(700)], dict(page=16, spare=0, short=100)),
    ([3 * i % 50 for i in range(700)], [i % 5 for i in range(700)], dict(page=16, spare=0, short=30)),
    ([0, 9], [5000, 4000], dict(page=16)),                     # more rows than a CTA's first pass
])
def test_take(seq, q, kw):
    x, geo = take_case(seq, q, **kw)
    got = run_take(seq, q, x["table"], x["stack"], x["count"], **geo)
    want = R.take(seq, q, x["table"], x["stack"], x["count"], **geo)
    assert got == tuple(want)


def test_take_with_bad_lengths():
    seq, q = [5, -3, 20, 30, 100, 10], [2, 1, -1, 9, 30, 3]
    table = [[i * 8 + j for j in range(8)] for i in range(6)]
    geo = dict(page=16, pages=60, rows=40, max_q=8, max_ctx=128)
    got = run_take(seq, q, table, list(range(48, 60)) + [0] * 48, 12, **geo)
    want = R.take(seq, q, table, list(range(48, 60)) + [0] * 48, 12, **geo)
    assert got == tuple(want) and want[4] & 1
    # rows that the call has no room for
    geo["rows"] = 4
    got = run_take([5, 6], [3, 3], table, list(range(48, 60)) + [0] * 48, 12, **geo)
    want = R.take([5, 6], [3, 3], table, list(range(48, 60)) + [0] * 48, 12, **geo)
    assert got == tuple(want) and want[4] == 1
    # a stack that says it holds more than the pool, or less than nothing
    for count in (61, -1):
        out = run_take([5], [1], table[:1], [0] * 60, count, **dict(geo, rows=1))
        assert out[4] == 1 and out[2] == [(0, 5, 5)]


def test_take_passes_on_page_numbers_that_are_none():
    geo = dict(page=16, pages=10, rows=20, max_q=20, max_ctx=64)
    got = run_take([0], [20], [[-1] * 4], [0, 1, 99, 3, 0, 0, 0, 0, 0, 0], 4, **geo)
    assert got[0] == [[3, 99, -1, -1]] and got[4] == 2
    assert [m[2] for m in got[2]] == list(range(48, 64)) + [-1] * 4


@pytest.mark.parametrize("kv", [B.PA_BF16, B.PA_MX4, B.PA_FP8_E4M3])
def test_take_without_rows_and_for_every_cache(kv):
    x, geo = take_case([5, 16], [0, 0], spare=4)
    geo["max_q"] = 1
    got = run_take([5, 16], [0, 0], x["table"], x["stack"], x["count"], kv=kv, **geo)
    assert got == (x["table"], [5, 16], [], x["count"], 0)


@pytest.mark.parametrize("seq,keep,page", [
    ([0], [0], 16), ([17], [16], 16), ([17], [0], 16), ([100, 33, 64], [100, 33, 64], 32),
    ([100, 33, 64], [97, 0, 1], 32), ([500, 5, 255], [3, 5, 0], 64),
    ([7 * i % 90 for i in range(1200)], [max(0, 7 * i % 90 - i % 40) for i in range(1200)], 16),
    ([100, 33, -1, 64, 2000], [101, 33, 0, -2, 0], 32),
])
def test_return(seq, keep, page):
    width = max(1, max(R.up(max(n, 0), page) for n in seq if n < 1000))
    total = sum(R.up(max(n, 0), page) for n in seq if n < 1000)
    pages = total + 9
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(3)).tolist()
    table, at = [], 0
    for n in seq:
        h = R.up(max(n, 0), page) if n < 1000 else width
        table.append((perm + perm)[at:at + h] + [-1] * (width - h))
        at += h if n < 1000 else 0
    if len(table) > 1 and len(seq) == 3 and page == 64:
        table[0][2] = -7                      # an entry that is none
    stack = perm[total:] + [-9] * total
    p = problem(num_seqs=len(seq), page_size=page, num_pages=pages, max_pages_per_seq=width,
                total_q_tokens=0, max_context_len=width * page)
    dev, left, err = ints(stack), ints([-9]), ints([0])
    B.pa_pages_return(p, ints(seq), ints(keep), ints(table), dev, ints([9]), left, err)
    want = R.give_back(seq, keep, table, stack, 9, page=page, pages=pages, max_ctx=width * page)
    assert (dev.tolist(), int(left), int(err)) == want


def test_return_past_the_stack():
    p = problem(num_seqs=2, num_pages=8, max_pages_per_seq=4, max_context_len=64)
    table = [[0, 1, 2, 3], [4, 5, 6, 7]]
    dev, left, err = ints([9] * 8 + [77] * 8), ints([0]), ints([0])
    B.pa_pages_return(p, ints([64, 64]), ints([0, 0]), ints(table), dev, ints([3]), left, err)
    assert dev.tolist() == [9] * 3 + [0, 1, 2, 3, 4] + [77] * 8
    assert int(left) == 8 and int(err) == 1


# -------------------------------------------------------------------- rope

def rope_case(T, Hq, Hkv, D, page, layout, kv, *, strided, seed, spare=2):
    g = torch.Generator().manual_seed(seed)
    width = (Hq + 2 * Hkv) * D + (24 if strided else 0)
    fused = torch.randn((T, width), generator=g).to(BF16).cuda()
    if strided:
        q, k, v = (fused[:, a * D:b * D].unflatten(1, (-1, D))
                   for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    else:
        q, k, v = (torch.randn((T, h, D), generator=g).to(BF16).cuda() for h in (Hq, Hkv, Hkv))
    pages = R.up(T, page) + spare
    slots = ints(torch.randperm(pages * page, generator=g)[:T].tolist())
    last = D if kv == B.PA_BF16 else D // 2
    shape = (pages, page, Hkv) if layout == 0 else (pages, Hkv, page)
    make = (lambda: torch.full((*shape, D), math.nan, dtype=BF16, device="cuda")) \
        if kv == B.PA_BF16 else (lambda: torch.full((*shape, last), 0xAA, dtype=torch.uint8,
                                                    device="cuda"))
    scales = [None, None] if kv == B.PA_BF16 else [
        torch.full((*shape, D // 32), 0xBB, dtype=torch.uint8, device="cuda") for _ in "kv"]
    p = problem(num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, page_size=page, num_pages=pages,
                max_pages_per_seq=pages, total_q_tokens=T, max_q_len=T,
                max_context_len=pages * page, layout=layout, kv_dtype=kv)
    return p, q, k, v, slots, make(), make(), scales


def cached(cache, slots, page, layout):
    s = slots.long()
    return cache[s // page, s % page] if layout == 0 else cache[s // page, :, s % page]


FREQ = torch.tensor([500000.0 ** (-i / 64) for i in range(64)], dtype=torch.float64)


def freq_of(rot):
    return FREQ[:: 128 // rot][:rot // 2] if 128 % rot == 0 else torch.tensor(
        [1e4 ** (-2 * i / rot) for i in range(rot // 2)], dtype=torch.float64)


@pytest.mark.parametrize("T,Hq,Hkv,D,page,layout,rot,inter,far,strided", [
    (1, 1, 1, 64, 16, 0, 64, 0, 0, False),
    (1, 8, 2, 128, 16, 1, 128, 1, 0, True),
    (3, 4, 1, 64, 32, 0, 16, 1, 5, True),
    (5, 7, 7, 128, 64, 1, 112, 0, 131071, False),
    (33, 32, 8, 128, 64, 0, 128, 0, 1000000, True),
    (33, 32, 8, 128, 64, 1, 64, 1, 2 ** 31 - 40, True),
    (64, 5, 1, 64, 128, 1, 48, 0, 77, True),
    (700, 3, 3, 64, 16, 0, 32, 1, 4096, False),
    (2500, 8, 1, 128, 256, 0, 96, 0, 123456, True),
    (6000, 16, 4, 128, 32, 1, 128, 1, 9, True),
])
def test_rope(T, Hq, Hkv, D, page, layout, rot, inter, far, strided):
    p, q, k, v, slots, kc, vc, _ = rope_case(T, Hq, Hkv, D, page, layout, B.PA_BF16,
                                             strided=strided, seed=T + rot)
    pos = ints([far + (i * 7) % 39 if i % 3 else (i * 13) % 50 for i in range(T)])
    rope = B.PaRope(rotary_dim=rot, interleaved=inter, cos_sin_scale=1.25 if T % 2 else 1.0)
    f, err = freq_of(rot), ints([0])
    out = torch.full((T, Hq, D), math.nan, dtype=BF16, device="cuda")
    before = kc.clone()
    B.pa_rope_append(p, rope, B.pa_rope_steps(f).cuda(), q, k, v, pos, slots, out, kc, None, vc,
                     None, err)
    no_error(err)
    for got, x in ((out, q), (cached(kc, slots, page, layout), k)):
        want, size = R.rotate(x.cpu(), pos.cpu(), f, rot, inter, rope.cos_sin_scale)
        # fp32: cos and sin off by 2^-24 of rounding, 2 ulp of sincospi and 2^-25 half turns of
        # angle, two products and a sum; then one rounding to bf16
        tol = HALF * want.abs() + size * (2.0 ** -24 * 6 + math.pi * 2.0 ** -25) * 1.01
        assert torch.all((got.cpu().double() - want).abs() <= tol)
        assert torch.equal(got.cpu()[..., rot:], x.cpu()[..., rot:])
    assert torch.equal(cached(vc, slots, page, layout), v)
    # nothing else was written
    touched = torch.zeros(before.shape[0] * page, dtype=torch.bool, device="cuda")
    touched[slots.long()] = True
    rest = ~touched.view(-1, page)
    for cache in (kc, vc):
        left = cache[rest] if layout == 0 else cache.transpose(1, 2)[rest]
        assert torch.isnan(left).all()


@pytest.mark.parametrize("D,rot,inter,layout,T", [(128, 128, 0, 0, 9), (128, 32, 0, 1, 40),
                                                  (64, 48, 0, 0, 7), (64, 64, 1, 1, 300),
                                                  (128, 112, 0, 1, 21), (64, 16, 1, 0, 2)])
def test_rope_into_a_4_bit_cache(D, rot, inter, layout, T):
    """Bit for bit what the bf16 cache's rows quantise to."""
    page, Hq, Hkv = 16, 4, 2
    f, rope = freq_of(rot), B.PaRope(rotary_dim=rot, interleaved=inter, cos_sin_scale=1.0)
    got = {}
    for kv in (B.PA_BF16, B.PA_MX4):
        p, q, k, v, slots, kc, vc, sc = rope_case(T, Hq, Hkv, D, page, layout, kv, strided=True,
                                                  seed=5)
        k[0, 0, 3] = math.inf                 # its block is NaN
        v[T - 1, 1] = 0.0
        k[T // 2, 1, D - 1] = 1e-38
        pos, err = ints(list(range(T))), ints([0])
        out = torch.zeros((T, Hq, D), dtype=BF16, device="cuda")
        B.pa_rope_append(p, rope, B.pa_rope_steps(f).cuda(), q, k, v, pos, slots, out, kc, sc[0],
                         vc, sc[1], err)
        no_error(err)
        got[kv] = [out] + [cached(x, slots, page, layout) for x in (kc, vc, *sc) if x is not None]
    assert torch.equal(got[B.PA_BF16][0].view(torch.int16), got[B.PA_MX4][0].view(torch.int16))
    for i in (1, 2):
        codes, scales = C.quantise(got[B.PA_BF16][i].cpu())
        assert torch.equal(got[B.PA_MX4][i].cpu(), codes)
        assert torch.equal(got[B.PA_MX4][i + 2].cpu(), scales)


def test_rope_rows_that_are_skipped():
    T, Hq, Hkv, D, page = 8, 2, 1, 128, 16
    p, q, k, v, slots, kc, vc, _ = rope_case(T, Hq, Hkv, D, page, 0, B.PA_BF16, strided=False,
                                             seed=1)
    steps, rope = B.pa_rope_steps(freq_of(128)).cuda(), B.PaRope(128, 0, 1.0)
    slots[2] = -1                             # padding
    pos, err = ints([3] * T), ints([0])
    out = torch.full((T, Hq, D), math.nan, dtype=BF16, device="cuda")
    B.pa_rope_append(p, rope, steps, q, k, v, pos, slots, out, kc, None, vc, None, err)
    no_error(err)
    skipped = torch.isnan(out).flatten(1).all(1)
    assert skipped.tolist() == [i == 2 for i in range(T)]
    assert int((~torch.isnan(kc)).flatten(2).all(2).sum()) == T - 1
    for bad, code in ((p.num_pages * page, 2), (2 ** 31 - 1, 2), (-2, 2)):
        s = slots.clone()
        s[5] = bad
        out.fill_(math.nan)
        err.zero_()
        B.pa_rope_append(p, rope, steps, q, k, v, pos, s, out, kc, None, vc, None, err)
        assert int(err) == code and torch.isnan(out).flatten(1).all(1).tolist() == [
            i in (2, 5) for i in range(T)]
    pos[4] = -1
    err.zero_()
    out.fill_(math.nan)
    B.pa_rope_append(p, rope, steps, q, k, v, pos, slots, out, kc, None, vc, None, err)
    assert int(err) == 1 and torch.isnan(out).flatten(1).all(1).tolist() == [
        i in (2, 4) for i in range(T)]


def test_rope_in_place_without_q_and_at_position_zero():
    T, Hq, Hkv, D, page = 40, 4, 2, 64, 16
    p, q, k, v, slots, kc, vc, _ = rope_case(T, Hq, Hkv, D, page, 1, B.PA_BF16, strided=False,
                                             seed=2)
    steps, rope = B.pa_rope_steps(freq_of(64)).cuda(), B.PaRope(64, 0, 1.0)
    pos, err = ints(list(range(100, 100 + T))), ints([0])
    out = torch.empty_like(q)
    B.pa_rope_append(p, rope, steps, q, k, v, pos, slots, out, kc, None, vc, None, err)
    k2, v2 = torch.full_like(kc, math.nan), torch.full_like(vc, math.nan)
    B.pa_rope_append(p, rope, steps, None, k, v, pos, slots, None, k2, None, v2, None, err)
    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))  # noqa: E731
    assert same(k2, kc) and same(v2, vc)
    qq = q.clone()
    B.pa_rope_append(p, rope, steps, qq, k, v, pos, slots, qq, k2, None, v2, None, err)
    assert same(qq, out)
    B.pa_rope_append(p, rope, steps, q, k, v, ints([0] * T), slots, out, kc, None, vc, None, err)
    assert same(out, q)                       # no turn at position 0
    no_error(err)


# ------------------------------------------------------------------ bounds

def new_slots(ctx, ql, page, pages, seed):
    """slots of the last ql[b] of ctx[b] tokens over shuffled pages, and the table."""
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table, slots, seq, pos, at = [], [], [], [], 0
    for b, (c, q) in enumerate(zip(ctx, ql)):
        row = perm[at:at + R.up(c, page)]
        at += R.up(c, page)
        table.append(row)
        for t in range(c - q, c):
            slots.append(row[t // page] * page + t % page)
            seq.append(b)
            pos.append(t)
    width = max(len(r) for r in table)
    return [r + [-1] * (width - len(r)) for r in table], slots, seq, pos


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx,ql,page,Hkv,layout,pad", [
    ([1], [1], 16, 1, 0, 0), ([16], [1], 16, 2, 1, 0), ([17, 40, 9], [1, 1, 1], 16, 3, 0, 2),
    ([200, 3], [200, 3], 32, 1, 1, 0), ([300, 70, 64, 1], [300, 70, 1, 0], 64, 4, 0, 5),
    ([700, 257], [600, 257], 256, 2, 1, 0), ([33] * 70, [2] * 70, 16, 2, 0, 0),
    ([5000], [5000], 128, 1, 0, 0),
])
def test_bounds(ctx, ql, page, Hkv, layout, pad, D):
    pages = sum(R.up(c, page) for c in ctx) + 2
    _, slots, _, _ = new_slots(ctx, ql, page, pages, 4)
    g = torch.Generator().manual_seed(D + page)
    k = torch.randn((pages, page, Hkv, D), generator=g) * torch.exp(
        2 * torch.randn((pages, 1, Hkv, D), generator=g))
    k = k.to(BF16)
    used = {}
    for s in slots:
        used[s // page] = s % page + 1
    for pg in range(pages):                   # what is behind the last key is not looked at
        k[pg, used.get(pg, 0):] = math.nan
    rows = len(slots) + pad
    p = problem(num_kv_heads=Hkv, num_q_heads=Hkv, head_dim=D, page_size=page, num_pages=pages,
                max_pages_per_seq=pages, total_q_tokens=rows, max_q_len=max(ql),
                max_context_len=pages * page, layout=layout)
    bnd = torch.full((pages, Hkv, 2, D), 99, dtype=torch.int8, device="cuda")
    sc, err = torch.full((pages, Hkv), -1.0, device="cuda"), ints([0])
    dev = (k if layout == 0 else k.transpose(1, 2)).contiguous().cuda()
    B.pa_page_bounds(p, dev, ints(slots + [-1] * pad), bnd, sc, err)
    no_error(err)
    for pg in range(pages):
        for h in range(Hkv):
            if pg not in used:
                assert torch.all(bnd[pg, h] == 99) and float(sc[pg, h]) == -1.0
                continue
            want, s = R.bounds(k[pg, :used[pg], h])
            assert float(sc[pg, h]) == s and torch.equal(bnd[pg, h].cpu(), want)


def test_bounds_of_odd_values():
    D, page = 64, 16
    rows = torch.zeros((9, page, 1, D))
    rows[1, :, 0, :] = 1e-30                  # below the least exponent's step
    rows[2, 3, 0, 5] = math.nan
    rows[2, 4, 0, 6] = 3.0
    rows[3, 3, 0, 5] = math.inf
    rows[3, 5, 0, 7] = -1e-30
    rows[4, 0, 0, 0], rows[4, 1, 0, 1] = 127.0, -127.0      # the largest of an exponent
    rows[5, 0, 0, 0] = 127.5                  # and the next number
    rows[6, 2, 0, 9] = -3e38
    rows[7, :, 0, :] = -0.0
    rows[8, 0, 0, 3] = -math.inf
    k = rows.to(BF16)
    p = problem(num_kv_heads=1, num_q_heads=1, head_dim=D, num_pages=9, max_pages_per_seq=9,
                total_q_tokens=9, max_q_len=9, max_context_len=144)
    bnd, sc = torch.zeros((9, 1, 2, D), dtype=torch.int8).cuda(), torch.zeros((9, 1)).cuda()
    err = ints([0])
    B.pa_page_bounds(p, k.cuda(), ints([i * 16 + 15 for i in range(9)]), bnd, sc, err)
    no_error(err)
    for i in range(9):
        want, s = R.bounds(k[i, :, 0])
        assert float(sc[i, 0]) == s, i
        assert torch.equal(bnd[i, 0].cpu(), want), i
    err.zero_()
    B.pa_page_bounds(p, k.cuda(), ints([144, -2, 2 ** 31 - 1] + [3] * 6), bnd, sc, err)
    assert int(err) == 2                      # the others are done


# --------------------------------------------------------------- selection

def random_bounds(pages, Hkv, D, seed):
    g = torch.Generator().manual_seed(seed)
    mid, half = torch.randn((pages, Hkv, D), generator=g), 2 + torch.rand((pages, Hkv, D), generator=g)
    top = (mid + half).abs().maximum((mid - half).abs()).amax(-1)
    e = torch.ceil(torch.log2(top / 127))
    unit = torch.exp2(e)[..., None]
    b = torch.stack((torch.ceil((mid + half) / unit), torch.floor((mid - half) / unit)), 2)
    return b.clamp(-127, 127).to(torch.int8), torch.exp2(e)


@pytest.mark.parametrize("D,G,Hkv,page,window,budget,first,recent,ctx,ql", [
    (128, 4, 2, 16, 0, 4, 1, 1, [1, 64, 65, 200], [1, 1, 1, 1]),
    (64, 1, 1, 16, 0, 1, 0, 0, [500, 3], [2, 1]),
    (128, 8, 1, 32, 0, 7, 2, 3, [3000, 100, 40], [1, 2, 0]),
    (64, 5, 3, 64, 0, 5, 0, 1, [2000, 321], [3, 1]),
    (128, 16, 1, 16, 0, 20, 1, 2, [4000], [1]),
    (128, 33, 1, 16, 0, 9, 1, 2, [900], [2]),
    (64, 64, 1, 32, 0, 3, 0, 0, [700, 90], [1, 1]),
    (128, 4, 2, 16, 500, 6, 1, 2, [2000, 200], [2, 1]),
    (64, 7, 2, 16, 17, 1, 0, 1, [300], [4]),
    (64, 2, 1, 16, 0, 300, 4, 20, [17000, 4800], [1, 1]),
    (128, 4, 8, 256, 0, 2, 0, 1, [1000] * 20, [1] * 20),
])
def test_selection(D, G, Hkv, page, window, budget, first, recent, ctx, ql):
    pages = sum(R.up(c, page) for c in ctx) + 2
    table, _, seq, pos = new_slots(ctx, ql, page, pages, 6)
    T = len(seq)
    bnd, sc = random_bounds(pages, Hkv, D, 7)
    q = torch.randn((T, G * Hkv, D), generator=torch.Generator().manual_seed(8)).to(BF16)
    p = problem(num_seqs=len(ctx), num_q_heads=G * Hkv, num_kv_heads=Hkv, head_dim=D,
                page_size=page, num_pages=pages, max_pages_per_seq=len(table[0]),
                total_q_tokens=T + 2, max_q_len=max(ql), max_context_len=max(ctx), window=window)
    sel, err = torch.full((T + 2, Hkv, budget), -7, dtype=torch.int32, device="cuda"), ints([0])
    qd = torch.cat((q, torch.full((2, G * Hkv, D), math.nan, dtype=BF16))).cuda()
    args = (qd, bnd.cuda(), sc.cuda(), ints(table), ints(seq + [-1, -1]), ints(pos + [0, 0]))
    B.pa_select_pages(p, budget, first, recent, *args, sel, err)
    no_error(err)
    assert torch.all(sel[T:] == -7)
    for t in range(T):
        for h in range(Hkv):
            want = R.select(q[t, h * G:(h + 1) * G], bnd[:, h], sc[:, h], table[seq[t]], pos[t],
                            budget=budget, num_first=first, num_recent=recent, page=page,
                            pages=pages, window=window)
            assert sel[t, h].tolist() == want, (t, h)


@pytest.mark.parametrize("D,G,page,n,budget", [(128, 3, 16, 90, 7), (64, 9, 32, 1500, 100),
                                               (128, 1, 16, 45056, 333)])
def test_selection_of_the_largest_sums_and_contexts(D, G, page, n, budget):
    """Codes of +-127 against queries of +-127: the largest whole numbers there are."""
    g = torch.Generator().manual_seed(n)
    bnd = torch.where(torch.rand((n, 1, 2, D), generator=g) < 0.5, 127, -127).to(torch.int8)
    bnd[: n // 2, :, 0], bnd[: n // 3, :, 1] = 127, -127
    bnd[n // 3:, :, :, 0] = torch.randint(-127, 128, (n - n // 3, 1, 2), generator=g).to(torch.int8)
    sc = torch.ones((n, 1))
    q = torch.where(torch.rand((2, G, D), generator=g) < 0.5, 127.0, -127.0).to(BF16)
    q[1, 0] = 127.0
    table = torch.randperm(n, generator=g).tolist()
    p = problem(num_q_heads=G, num_kv_heads=1, head_dim=D, page_size=page, num_pages=n,
                max_pages_per_seq=n, total_q_tokens=2, max_q_len=2, max_context_len=n * page)
    sel, err = torch.zeros((2, 1, budget), dtype=torch.int32, device="cuda"), ints([0])
    B.pa_select_pages(p, budget, 2, 3, q.cuda(), bnd.cuda(), sc.cuda(), ints([table]),
                      ints([0, 0]), ints([n * page - 1] * 2), sel, err)
    no_error(err)
    for t in range(2):
        b = bnd[torch.tensor(table), 0].double()
        # (some of these bounds have the smallest above the largest, where the larger of the
        # two products is not the definition's)
        c = q[t].double()[:, None]
        score = (c * torch.where(c > 0, b[None, :, 0], b[None, :, 1])).sum(-1).amax(0)
        score[:2] = score[-3:] = math.inf
        want = torch.sort(score, descending=True, stable=True)[1][:budget].sort()[0]
        assert sel[t, 0].tolist() == want.tolist()


def test_selection_of_ties_odd_queries_and_bad_pages():
    D, page, n, budget = 64, 16, 200, 8
    table = list(range(n))
    bnd, sc = random_bounds(n, 1, D, 1)
    bnd[:], sc[:] = bnd[0], sc[0]             # every page the same: the lowest ones
    q = torch.randn((6, 2, D), generator=torch.Generator().manual_seed(2)).to(BF16)
    q[1] = 0.0
    q[2, 0, 5], q[2, 1, :] = math.nan, math.nan
    q[3, 1, 7] = -math.inf
    q[4] = 3e38
    q[5] = 1e-38
    bnd[150, 0, 0], sc[60] = 127, 2.0 ** 40
    table[10], table[199], table[0] = -1, 777, n
    p = problem(num_q_heads=2, num_kv_heads=1, head_dim=D, num_pages=n, max_pages_per_seq=n,
                total_q_tokens=6, max_q_len=6, max_context_len=n * page)
    sel, err = torch.zeros((6, 1, budget), dtype=torch.int32, device="cuda"), ints([0])
    B.pa_select_pages(p, budget, 0, 2, q.cuda(), bnd.cuda(), sc.cuda(), ints([table]),
                      ints([0] * 6), ints([n * page - 1] * 6), sel, err)
    assert int(err) == 2
    for t in range(6):
        want = R.select(q[t], bnd[:, 0], sc[:, 0], table, n * page - 1, budget=budget, num_first=0,
                        num_recent=2, page=page, pages=n, window=0)
        assert sel[t, 0].tolist() == want, t
    # a page whose scale is none is the last to be listed
    odd = sc.clone()
    odd[3], odd[7, 0], odd[100] = math.nan, -1.0, math.inf
    got = torch.full_like(sel, -3)
    B.pa_select_pages(p, budget, 0, 2, q.cuda(), bnd.cuda(), odd.cuda(), ints([table]),
                      ints([0] * 6), ints([n * page - 1] * 6), got, err)
    for t in range(6):
        row = got[t, 0].tolist()
        assert row == sorted(set(row)) and 0 <= row[0] and row[-2:] == [n - 2, n - 1]
        assert 3 not in row and 7 not in row
    # the cache's type has no part in it
    for kv in (B.PA_FP8_E4M3, B.PA_MX4):
        p.kv_dtype = kv
        again = torch.zeros_like(sel)
        B.pa_select_pages(p, budget, 0, 2, q.cuda(), bnd.cuda(), sc.cuda(), ints([table]),
                          ints([0] * 6), ints([n * page - 1] * 6), again, err)
        assert torch.equal(again, sel)
    # rows that cannot be: left as they are
    sel.fill_(-5)
    err.zero_()
    B.pa_select_pages(p, budget, 0, 2, q.cuda(), bnd.cuda(), sc.cuda(), ints([table]),
                      ints([0, 1, -1, 0, 0, 0]), ints([5, 5, 5, -1, n * page, 31]), sel, err)
    assert int(err) == 1
    assert [bool((sel[t] == -5).all()) for t in range(6)] == [False, True, True, True, True, False]
    assert sel[5, 0].tolist() == [0, 1] + [-1] * 6


# --------------------------------------------------------------- attention

def attend_case(D, G, Hkv, page, layout, ctx, ql, seed, spare=2, mag=1.0):
    pages = sum(R.up(c, page) for c in ctx) + spare
    table, _, seq, pos = new_slots(ctx, ql, page, pages, seed)
    g = torch.Generator().manual_seed(seed + 1)
    k = (torch.randn((pages, page, Hkv, D), generator=g) * mag).to(BF16)
    v = torch.randn((pages, page, Hkv, D), generator=g).to(BF16)
    q = torch.randn((len(seq), G * Hkv, D), generator=g).to(BF16)
    return pages, table, seq, pos, k, v, q


def check_attend(p, budget, table, seq, pos, k, v, q, sel, code=0, repeat=1):
    """Runs the call and compares every row of a sequence; the others stay as they are."""
    T, H, D = q.shape
    Hkv, page, pages = p.num_kv_heads, p.page_size, p.num_pages
    G, layout = H // Hkv, p.layout
    dev = [(x if layout == 0 else x.transpose(1, 2)).contiguous().cuda() for x in (k, v)]
    ws = torch.zeros(B.pa_selected_workspace_size(p, budget), dtype=torch.uint8, device="cuda")
    out = torch.full((T, H, D), 7.0, dtype=BF16, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    args = (q.cuda(), *dev, ints(table), ints(seq), ints(pos), ints(sel), ws)
    for _ in range(repeat):
        B.pa_decode_selected(p, budget, *args, out, lse)
    assert B.pa_last_device_error(ws) == code
    assert not ws[256:256 + 1024 * 64 * 4].any()   # the counters as the next call finds them
    for t in range(T):
        if not (0 <= seq[t] < p.num_seqs and 0 <= pos[t] < p.max_context_len):
            assert torch.all(out[t] == 7) and torch.all(lse[t] == 7)
            continue
        first, n = R.seen_pages(pos[t], page, p.window)
        for h in range(Hkv):
            ks, vs, at = [], [], []
            for s in sel[t][h][:min(budget, n)]:
                if not 0 <= s <= pos[t] // page:
                    continue
                pg = table[seq[t]][s]
                if 0 <= pg < pages:
                    ks.append(k[pg, :, h])
                    vs.append(v[pg, :, h])
                    at += range(s * page, s * page + page)
            kk = torch.cat(ks) if ks else torch.zeros((0, D))
            vv = torch.cat(vs) if vs else torch.zeros((0, D))
            r = slice(h * G, (h + 1) * G)
            o, L, size, big = R.attend(q[t, r], kk, vv, at, pos[t], p.window, p.sm_scale)
            # scores in fp32 sums of D products; probabilities and the result rounded to bf16
            ds = (D + 16) * 2.0 ** -24 * big[:, None] + 2.0 ** -20
            tol = (HALF + 2 * ds) * size * 1.01 + HALF * (o.abs() + HALF * size)
            assert torch.all((out[t, r].cpu().double() - o).abs() <= tol), (t, h)
            got = lse[t, r].cpu().double()
            none = torch.isinf(L)
            assert torch.equal(got[none], L[none])
            far = (got - L).abs()[~none]
            assert torch.all(far <= (ds[:, 0] + 2.0 ** -22 * (1 + L.abs()))[~none]), (t, h)
    return out, lse


def lists(seq, pos, Hkv, budget, page, window, seed, mode="plain"):
    g = torch.Generator().manual_seed(seed)
    out = []
    for s, x in zip(seq, pos):
        first, n = R.seen_pages(max(x, 0), page, window)
        rows = []
        for _ in range(Hkv):
            got = (first + torch.randperm(n, generator=g)[:budget].sort()[0]).tolist()
            if mode == "holes":
                got = [y if i % 3 else -1 for i, y in enumerate(got)]
            elif mode == "shuffled":
                got = got[::-1]
            elif mode == "twice":
                got = (got + got)[:min(budget, n)] if len(got) < budget else got[:-1] + got[:1]
            elif mode == "none":
                got = [-1] * len(got)
            rows.append(got + [-1] * (budget - len(got)))
        out.append(rows)
    return out


@pytest.mark.parametrize("ctas", [0, 1, 5, 700])
@pytest.mark.parametrize("D,G,Hkv,page,layout,window,budget,ctx,ql,mode", [
    (128, 4, 2, 16, 0, 0, 4, [1, 64, 65, 200], [1, 1, 1, 1], "plain"),
    (64, 1, 1, 16, 1, 0, 1, [500, 3], [2, 1], "plain"),
    (128, 8, 1, 64, 1, 0, 9, [3000, 100, 40], [1, 2, 0], "plain"),
    (64, 5, 3, 64, 0, 0, 5, [2000, 321], [3, 1], "holes"),
    (128, 16, 1, 16, 0, 0, 20, [4000], [1], "shuffled"),
    (128, 29, 1, 32, 1, 0, 9, [900], [2], "plain"),
    (64, 64, 1, 32, 0, 0, 3, [700, 90], [1, 1], "plain"),
    (64, 30, 2, 16, 1, 0, 30, [700, 90], [1, 1], "holes"),
    (64, 9, 2, 16, 1, 0, 40, [700, 90], [1, 1], "plain"),
    (128, 4, 2, 16, 0, 500, 40, [2000, 200], [2, 1], "plain"),
    (64, 7, 2, 16, 0, 17, 2, [300], [4], "plain"),
    (128, 4, 2, 128, 0, 0, 3, [1000, 129], [1, 1], "twice"),
    (128, 2, 1, 256, 1, 100, 6, [1025, 200], [2, 1], "plain"),
    (64, 2, 1, 16, 0, 0, 900, [17000, 4800], [1, 1], "plain"),
    (128, 3, 2, 16, 0, 0, 5, [100, 20], [1, 1], "none"),
])
def test_attention(D, G, Hkv, page, layout, window, budget, ctx, ql, mode, ctas):
    pages, table, seq, pos, k, v, q = attend_case(D, G, Hkv, page, layout, ctx, ql, 3)
    sel = lists(seq, pos, Hkv, budget, page, window, 5, mode)
    # what no row may see is NaN: pages that nobody lists, and keys behind the last position
    listed = set()
    for t in range(len(seq)):
        for h in range(Hkv):
            listed |= {(table[seq[t]][s], h) for s in sel[t][h] if s >= 0}
    for pg in range(pages):
        for h in range(Hkv):
            if (pg, h) not in listed:
                k[pg, :, h] = v[pg, :, h] = math.nan
    for b, c in enumerate(ctx):
        if c % page:
            pg = table[b][c // page]
            k[pg, c % page:] = v[pg, c % page:] = math.nan
    p = problem(num_seqs=len(ctx), num_q_heads=G * Hkv, num_kv_heads=Hkv, head_dim=D,
                page_size=page, num_pages=pages, max_pages_per_seq=len(table[0]), layout=layout,
                total_q_tokens=len(seq), max_q_len=max(ql), max_context_len=max(ctx),
                window=window, num_ctas=ctas, sm_scale=1.0 / math.sqrt(D))
    check_attend(p, budget, table, seq, pos, k, v, q, sel, repeat=2)


@pytest.mark.parametrize("ctas", [0, 3])
@pytest.mark.parametrize("D,G,Hkv,page,layout,window,budget,ctx,ql,mode", [
    (128, 1, 2, 16, 0, 0, 5, [400, 90, 13], [13, 6, 13], "plain"),
    (128, 4, 2, 16, 1, 0, 7, [400, 90, 7], [4, 0, 7], "plain"),
    (128, 7, 1, 32, 0, 100, 6, [700, 65], [4, 3], "holes"),
    (128, 8, 2, 64, 1, 0, 4, [2000, 70, 300], [3, 3, 2], "shuffled"),
    (128, 16, 1, 16, 0, 0, 9, [500, 33], [2, 5], "plain"),
    (64, 2, 3, 16, 0, 17, 2, [300, 40], [9, 9], "plain"),
    (64, 5, 1, 128, 1, 0, 3, [1500, 130], [6, 4], "plain"),
    (64, 11, 1, 16, 0, 0, 40, [700, 90], [2, 1], "plain"),
    (64, 20, 2, 32, 0, 0, 4, [700, 90], [3, 1], "plain"),
    (64, 1, 1, 16, 0, 0, 50, [70000, 90], [5, 1], "plain"),
    (128, 3, 2, 16, 0, 0, 5, [100, 20], [3, 2], "none"),
    (64, 4, 1, 16, 0, 0, 6, [300, 9], [300, 9], "plain"),
])
def test_attention_of_rows_of_one_sequence(D, G, Hkv, page, layout, window, budget, ctx, ql, mode,
                                           ctas):
    pages, table, seq, pos, k, v, q = attend_case(D, G, Hkv, page, layout, ctx, ql, 3)
    sel = lists(seq, pos, Hkv, budget, page, window, 5, mode)
    for t in range(1, len(seq)):              # rows of a sequence share some of their pages
        if seq[t] == seq[t - 1] and t % 3:
            sel[t] = [list(x) for x in sel[t - 1]]
    listed = {(table[seq[t]][s], h) for t in range(len(seq)) for h in range(Hkv)
              for s in sel[t][h] if s >= 0}
    for pg in range(pages):
        for h in range(Hkv):
            if (pg, h) not in listed:
                k[pg, :, h] = v[pg, :, h] = math.nan
    p = problem(num_seqs=len(ctx), num_q_heads=G * Hkv, num_kv_heads=Hkv, head_dim=D,
                page_size=page, num_pages=pages, max_pages_per_seq=len(table[0]), layout=layout,
                total_q_tokens=len(seq), max_q_len=max(ql), max_context_len=max(ctx),
                window=window, num_ctas=ctas, sm_scale=1.0 / math.sqrt(D))
    check_attend(p, budget, table, seq, pos, k, v, q, sel, repeat=2)


def test_what_one_row_lists_does_not_reach_its_neighbour():
    """Infinities and NaN in a page that only one of two rows lists, and in the later row's
    own token."""
    for D, G, page in ((128, 4, 16), (64, 3, 32), (128, 12, 64)):
        pages, table, seq, pos, k, v, q = attend_case(D, G, 1, page, 0, [520], [2], 9)
        n = R.up(520, page)
        sel = [[[0, 2, 3, n - 1]], [[0, 1, 3, n - 1]]]
        p = problem(num_q_heads=G, num_kv_heads=1, head_dim=D, page_size=page, num_pages=pages,
                    max_pages_per_seq=n, total_q_tokens=2, max_q_len=2, max_context_len=520)
        good, glse = check_attend(p, 4, table, seq, pos, k, v, q, sel)
        ws = torch.zeros(B.pa_selected_workspace_size(p, 4), dtype=torch.uint8, device="cuda")
        for value in (math.inf, -math.inf, math.nan):
            for which in ("k", "v"):
                for pg, slot, hit in ((table[0][1], 5, 1), (table[0][2], 9, 0),
                                      (table[0][n - 1], 519 % page, 1)):
                    k2, v2 = k.clone(), v.clone()
                    (k2 if which == "k" else v2)[pg, slot, 0, 7] = value
                    out, lse = torch.zeros_like(good), torch.zeros_like(glse)
                    B.pa_decode_selected(p, 4, q.cuda(), k2.cuda(), v2.cuda(), ints(table),
                                         ints(seq), ints(pos), ints(sel), ws, out, lse)
                    miss = 1 - hit
                    # (the same sums but for how a step's products are grouped)
                    assert float((out[miss].float() - good[miss].float()).abs().max()) <= 2e-2
                    assert float((lse[miss] - glse[miss]).abs().max()) <= 1e-3
                    if which == "v":
                        bad = ~torch.isfinite(out[hit])
                        assert bad[:, 7].all() and not bad[:, :7].any() and not bad[:, 8:].any()
                    elif value != value:
                        assert torch.isnan(out[hit]).all()


def test_attention_past_bad_entries():
    D, G, Hkv, page, budget = 128, 2, 1, 16, 6
    pages, table, seq, pos, k, v, q = attend_case(D, G, Hkv, page, 0, [300, 200, 64], [1, 1, 1], 9)
    sel = lists(seq, pos, Hkv, budget, page, 0, 5)
    p = problem(num_seqs=3, num_q_heads=G, num_kv_heads=Hkv, num_pages=pages,
                max_pages_per_seq=len(table[0]), total_q_tokens=6, max_q_len=1,
                max_context_len=300)
    q = torch.cat((q, q))
    rows = dict(seq=seq + [-1, 3, 0], pos=pos + [0, 5, 300])
    sel = sel + sel
    # padding is no error, a sequence or position that cannot be is one
    check_attend(p, budget, table, k=k, v=v, q=q, sel=sel, code=1, **rows)
    rows = dict(seq=seq + [-1] * 3, pos=pos + [0] * 3)
    check_attend(p, budget, table, k=k, v=v, q=q, sel=sel, **rows)
    bad = [[list(x) for x in r] for r in sel]
    bad[0][0][2] = 19                         # behind the row's own page
    check_attend(p, budget, table, k=k, v=v, q=q, sel=bad, code=1, **rows)
    bad[0][0][2] = -2 ** 31
    check_attend(p, budget, table, k=k, v=v, q=q, sel=bad, code=1, **rows)
    t2 = [list(r) for r in table]
    t2[1][sel[1][0][1]], t2[1][sel[1][0][3]] = -1, pages
    check_attend(p, budget, t2, k=k, v=v, q=q, sel=sel, code=2, **rows)


def test_attention_with_large_scores_infinities_and_nan():
    D, G, Hkv, page, budget = 128, 4, 1, 16, 8
    pages, table, seq, pos, k, v, q = attend_case(D, G, Hkv, page, 0, [500, 400], [1, 1], 9, mag=30)
    sel = lists(seq, pos, Hkv, budget, page, 0, 5)
    p = problem(num_seqs=2, num_q_heads=G, num_kv_heads=Hkv, num_pages=pages,
                max_pages_per_seq=len(table[0]), total_q_tokens=2, max_q_len=1,
                max_context_len=500, sm_scale=1.0)
    check_attend(p, budget, table, seq, pos, k, v, q, sel)       # one key outweighs the rest
    # the first list's first page: an infinite V element reaches its column alone, a NaN key all
    ws = torch.zeros(B.pa_selected_workspace_size(p, budget), dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros((2, G, D), dtype=BF16, device="cuda"), torch.zeros((2, G)).cuda()
    p.sm_scale = 0.001
    v2, k2 = v.clone(), k.clone()
    v2[table[0][sel[0][0][0]], 3, 0, 11] = math.inf
    call = lambda kk, vv: B.pa_decode_selected(  # noqa: E731
        p, budget, q.cuda(), kk.cuda(), vv.cuda(), ints(table), ints(seq), ints(pos), ints(sel),
        ws, out, lse)
    call(k, v2)
    assert torch.isinf(out[0, :, 11]).all() and torch.isfinite(out[1]).all()
    assert torch.isfinite(out[0, :, :11]).all() and torch.isfinite(out[0, :, 12:]).all()
    k2[table[0][sel[0][0][0]], 3, 0, 5] = math.nan
    call(k2, v)
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all() and torch.isfinite(out[1]).all()
    # nor does what the row does not list reach it
    p.sm_scale = 0.1
    call(k, v)
    before = out.clone()
    unlisted = next(s for s in range(20) if s not in sel[0][0])
    k2 = k.clone()
    k2[table[0][unlisted]] = v[table[0][unlisted]] = math.inf
    call(k2, v)
    assert torch.equal(out, before)


def test_attention_is_pa_decode_where_every_page_is_listed():
    """All pages listed: the softmax over the whole context, against the oracle's kernel."""
    D, G, Hkv, page = 128, 4, 2, 64
    ctx, ql = [1000, 64, 333], [2, 2, 2]
    pages, table, seq, pos, k, v, q = attend_case(D, G, Hkv, page, 0, ctx, ql, 13)
    budget = 16
    sel = lists(seq, pos, Hkv, budget, page, 0, 5)
    p = problem(num_seqs=3, num_q_heads=G * Hkv, num_kv_heads=Hkv, page_size=page, num_pages=pages,
                max_pages_per_seq=len(table[0]), total_q_tokens=6, max_q_len=2,
                max_context_len=1000)
    out, lse = check_attend(p, budget, table, seq, pos, k, v, q, sel)
    a = torch.empty(B.pa_assign_workspace_size(p, 0), dtype=torch.uint8, device="cuda")
    w = torch.empty(B.pa_partial_workspace_size(p, 0), dtype=torch.uint8, device="cuda")
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    c, n, t = ints(ctx), ints(ql), ints(table)
    B.pa_assign(p, 0, c, n, None, a)
    B.pa_decode_splitk(p, q.cuda(), k.cuda(), v.cuda(), t, c, n, None, None, a, w, o2, l2)
    B.pa_combine(p, 0, a, w, o2, l2)
    assert float((out.float() - o2.float()).abs().max()) <= 2e-2
    assert float((lse - l2).abs().max()) <= 1e-3


def test_one_workspace_for_calls_of_other_shapes():
    """Calls of other grids, groups and rows a sequence follow one another in one workspace."""
    cases = [(128, 4, 2, 16, [500, 90], [1, 1], 7, 0), (64, 16, 1, 32, [900], [1], 20, 1000),
             (128, 3, 1, 16, [700, 30], [4, 2], 9, 17), (128, 8, 1, 16, [2000], [1], 100, 300)]
    ps = []
    for D, G, Hkv, page, ctx, ql, budget, ctas in cases:
        c = attend_case(D, G, Hkv, page, 0, ctx, ql, 3)
        p = problem(num_seqs=len(ctx), num_q_heads=G * Hkv, num_kv_heads=Hkv, head_dim=D,
                    page_size=page, num_pages=c[0], max_pages_per_seq=len(c[1][0]),
                    total_q_tokens=len(c[2]), max_q_len=max(ql), max_context_len=max(ctx),
                    num_ctas=ctas)
        ps.append((p, budget, c, lists(c[2], c[3], Hkv, budget, page, 0, 5)))
    need = max(B.pa_selected_workspace_size(p, budget) for p, budget, _, _ in ps)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        for p, budget, (_, table, seq, pos, k, v, q), sel in ps:
            want, wl = check_attend(p, budget, table, seq, pos, k, v, q, sel)
            out, lse = torch.zeros_like(want), torch.zeros_like(wl)
            B.pa_decode_selected(p, budget, q.cuda(), k.cuda(), v.cuda(), ints(table), ints(seq),
                                 ints(pos), ints(sel), ws, out, lse)
            assert B.pa_last_device_error(ws) == 0
            assert torch.equal(out, want) and torch.equal(lse, wl)


def test_pages_past_2_to_the_32_bytes():
    """Rope, bounds and attention on the last pages of caches of more than 2^32 bytes (and of
    more than 2^31 elements)."""
    D, Hkv, G, page = 128, 8, 2, 64
    pages = (2 ** 32 // (page * Hkv * D * 2)) + 40
    k = torch.zeros((pages, page, Hkv, D), dtype=BF16, device="cuda")
    v = torch.zeros_like(k)
    assert k.numel() > 2 ** 31
    n = 150
    table = ints([[pages - 1, 0, pages - 2]])
    p = problem(num_q_heads=G * Hkv, num_kv_heads=Hkv, page_size=page, num_pages=pages,
                max_pages_per_seq=3, total_q_tokens=n, max_q_len=n, max_context_len=192)
    g = torch.Generator().manual_seed(3)
    q, kn, vn = (torch.randn((n, h, D), generator=g).to(BF16).cuda() for h in (G * Hkv, Hkv, Hkv))
    pos = ints(list(range(n)))
    slots = (table[0].long()[pos.long() // page] * page + pos % page).int()
    err, out = ints([0]), torch.zeros_like(q)
    B.pa_rope_append(p, B.PaRope(16, 0, 1.0), B.pa_rope_steps(torch.zeros(8)).cuda(), q, kn, vn, pos,
                     slots, out, k, None, v, None, err)
    s = slots.long()
    assert torch.equal(k[s // page, s % page], kn) and torch.equal(v[s // page, s % page], vn)
    assert int(torch.count_nonzero(k[1:pages - 2])) == 0
    bnd = torch.zeros((pages, Hkv, 2, D), dtype=torch.int8, device="cuda")
    sc = torch.zeros((pages, Hkv), device="cuda")
    B.pa_page_bounds(p, k, slots, bnd, sc, err)
    no_error(err)
    for i, used in ((0, 64), (1, 64), (2, 22)):
        for h in (0, Hkv - 1):
            want, scale = R.bounds(kn[i * page:i * page + used, h].cpu())
            pg = int(table[0, i])
            assert float(sc[pg, h]) == scale and torch.equal(bnd[pg, h].cpu(), want)
    p.total_q_tokens, p.max_q_len = 1, 1
    sel = ints([[[0, 1, 2]] * Hkv])
    ws = torch.zeros(B.pa_selected_workspace_size(p, 3), dtype=torch.uint8, device="cuda")
    o, lse = torch.zeros((1, G * Hkv, D), dtype=BF16, device="cuda"), torch.zeros((1, G * Hkv)).cuda()
    B.pa_decode_selected(p, 3, q, k, v, table, ints([0]), ints([n - 1]), sel, ws, o, lse)
    for h in range(Hkv):
        r = slice(h * G, (h + 1) * G)
        want, L, size, big = R.attend(q[0, r].cpu(), kn[:, h].cpu(), vn[:, h].cpu(), list(range(n)),
                                      n - 1, 0, p.sm_scale)
        ds = (D + 16) * 2.0 ** -24 * big[:, None] + 2.0 ** -20
        tol = (HALF + 2 * ds) * size * 1.01 + HALF * (want.abs() + HALF * size)
        assert torch.all((o[0, r].cpu().double() - want).abs() <= tol)


def test_a_workspace_that_was_never_filled_is_reported():
    D, G, Hkv, page, budget = 64, 1, 1, 16, 64
    pages, table, seq, pos, k, v, q = attend_case(D, G, Hkv, page, 0, [1024], [1], 9)
    sel = lists(seq, pos, Hkv, budget, page, 0, 5)
    p = problem(num_q_heads=1, num_kv_heads=1, head_dim=D, num_pages=pages, max_pages_per_seq=64,
                max_context_len=1024, num_ctas=5)
    ws = torch.zeros(B.pa_selected_workspace_size(p, budget), dtype=torch.uint8, device="cuda")
    ws[256:256 + 1024 * 64 * 4] = 1
    out, lse = torch.zeros((1, 1, D), dtype=BF16, device="cuda"), torch.zeros((1, 1)).cuda()
    args = (q.cuda(), k.cuda(), v.cuda(), ints(table), ints(seq), ints(pos), ints(sel), ws)
    B.pa_decode_selected(p, budget, *args, out, lse)
    assert B.pa_last_device_error(ws) == B.PA_DEV_BAD_WORKSPACE
    ws.zero_()
    check_attend(p, budget, table, seq, pos, k, v, q, sel)


# ------------------------------------------------------------ all together

class Loop:
    """A decode loop over a paged cache as a server runs it, all state on the GPU."""

    def __init__(self, B_, Hq, Hkv, D, page, layout, budget, rows, max_ctx, seed=0):
        self.p = problem(num_seqs=B_, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, page_size=page,
                         num_pages=B_ * R.up(max_ctx, page) + 3, layout=layout,
                         max_pages_per_seq=R.up(max_ctx, page), total_q_tokens=rows,
                         max_q_len=rows, max_context_len=max_ctx, sm_scale=1 / math.sqrt(D))
        n = self.p.num_pages
        shape = (n, page, Hkv, D) if layout == 0 else (n, Hkv, page, D)
        self.k, self.v = (torch.full(shape, math.nan, dtype=BF16, device="cuda") for _ in "kv")
        self.bnd = torch.zeros((n, Hkv, 2, D), dtype=torch.int8, device="cuda")
        self.sc = torch.zeros((n, Hkv), device="cuda")
        self.table = torch.full((B_, self.p.max_pages_per_seq), -1, dtype=torch.int32).cuda()
        self.free = ints(torch.randperm(n, generator=torch.Generator().manual_seed(seed)).tolist())
        self.count, self.left = ints([n]), ints([0])
        self.lens, self.ctx, self.ql = ints([0] * B_), ints([0] * B_), ints([0] * B_)
        self.seq, self.pos, self.slots = (ints([0] * rows) for _ in range(3))
        self.budget = budget
        self.sel = torch.zeros((rows, Hkv, budget), dtype=torch.int32, device="cuda")
        self.ws = torch.zeros(B.pa_selected_workspace_size(self.p, budget), dtype=torch.uint8,
                              device="cuda")
        self.qr, self.out = (torch.zeros((rows, Hq, D), dtype=BF16, device="cuda") for _ in "ab")
        self.lse, self.err = torch.zeros((rows, Hq), device="cuda"), ints([0])
        self.freq = freq_of(D)
        self.steps, self.rope = B.pa_rope_steps(self.freq).cuda(), B.PaRope(D, 0, 1.0)
        self.fused = torch.zeros((rows, (Hq + 2 * Hkv) * D), dtype=BF16, device="cuda")
        self.q, self.kn, self.vn = (x.unflatten(1, (-1, D)) for x in self.fused.split(
            [Hq * D, Hkv * D, Hkv * D], 1))

    def step(self):
        p = self.p
        B.pa_pages_take(p, self.lens, self.ql, self.table, self.free, self.count, self.ctx,
                        self.seq, self.pos, self.slots, self.left, self.err)
        B.pa_rope_append(p, self.rope, self.steps, self.q, self.kn, self.vn, self.pos, self.slots,
                         self.qr, self.k, None, self.v, None, self.err)
        B.pa_page_bounds(p, self.k, self.slots, self.bnd, self.sc, self.err)
        B.pa_select_pages(p, self.budget, 1, 1, self.qr, self.bnd, self.sc, self.table, self.seq,
                          self.pos, self.sel, self.err)
        B.pa_decode_selected(p, self.budget, self.qr, self.k, self.v, self.table, self.seq,
                             self.pos, self.sel, self.ws, self.out, self.lse)
        self.count.copy_(self.left)
        self.lens.copy_(self.ctx)

    def give_back(self, keep):
        B.pa_pages_return(self.p, self.lens, keep, self.table, self.free, self.count, self.left,
                          self.err)
        self.count.copy_(self.left)
        self.lens.copy_(keep)


@pytest.mark.parametrize("Hq,Hkv,D,page,layout,graph", [(8, 2, 128, 16, 0, False),
                                                        (5, 5, 64, 32, 1, True),
                                                        (16, 2, 64, 16, 0, True)])
def test_a_decode_loop(Hq, Hkv, D, page, layout, graph):
    """Prompts, decode steps, drafts taken back and a finished sequence's pages used again,
    with one captured step replayed; every step against the definition over the whole history."""
    N, rows, budget, max_ctx = 3, 24, 5, 320
    L = Loop(N, Hq, Hkv, D, page, layout, budget, rows, max_ctx)
    g = torch.Generator().manual_seed(1)
    G = Hq // Hkv
    hist = [[] for _ in range(N)]                      # (rotated key, value) of every token
    run = L.step
    if graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            L.step()                                   # nothing new: no row, no page
        torch.cuda.current_stream().wait_stream(side)
        G_ = torch.cuda.CUDAGraph()
        with torch.cuda.graph(G_):
            L.step()
        run = G_.replay
    plan = [[20, 1, 0], [20, 3, 1]] + [[22, 1, 1]] * 10 + [[1, 1, 1]] * 8 + [[3, 3, 3]] * 4
    for i, ql in enumerate(plan):
        if i in (8, 15):
            # drafts of sequence 0 not accepted; sequence 1 done
            keep = [len(h) for h in hist]
            keep[0] -= 3
            keep[1] = 0 if i == 15 else keep[1]
            L.give_back(ints(keep))
            hist = [h[:n] for h, n in zip(hist, keep)]
        x = torch.randn(L.fused.shape, generator=g).to(BF16)
        L.fused.copy_(x)
        L.ql.copy_(ints(ql))
        L.out.fill_(7.0)
        run()
        assert int(L.err) == 0 and B.pa_last_device_error(L.ws) == 0
        q, kn, vn = L.q.cpu(), L.kn.cpu(), L.vn.cpu()
        t = 0
        kd = L.k.cpu() if layout == 0 else L.k.cpu().transpose(1, 2)
        table, sel = L.table.tolist(), L.sel.tolist()
        for b, n in enumerate(ql):
            for _ in range(n):
                pos = len(hist[b])
                slot = table[b][pos // page] * page + pos % page
                k_here = kd[slot // page, slot % page]
                want, size = R.rotate(kn[t:t + 1], torch.tensor([pos]), L.freq, D, 0, 1.0)
                assert torch.all((k_here.double() - want[0]).abs()
                                 <= HALF * want[0].abs() + size[0] * 5e-7)
                hist[b].append((k_here, vn[t]))
                t += 1
        t = 0
        bnd, sc = L.bnd.cpu(), L.sc.cpu()
        qr, out = L.qr.cpu(), L.out.cpu()
        for b, n in enumerate(ql):
            for j in range(n):
                pos = len(hist[b]) - n + j
                for h in range(Hkv):
                    r = slice(h * G, (h + 1) * G)
                    want = R.select(qr[t, r], bnd[:, h], sc[:, h], table[b], pos, budget=budget,
                                    num_first=1, num_recent=1, page=page, pages=L.p.num_pages,
                                    window=0)
                    assert sel[t][h] == want
                    at = [x for s in want if s >= 0 for x in range(s * page, min(s * page + page, pos + 1))]
                    kk = torch.stack([hist[b][x][0][h] for x in at])
                    vv = torch.stack([hist[b][x][1][h] for x in at])
                    o, _, size, big = R.attend(qr[t, r], kk, vv, at, pos, 0, L.p.sm_scale)
                    ds = (D + 16) * 2.0 ** -24 * big[:, None] + 2.0 ** -20
                    tol = (HALF + 2 * ds) * size * 1.01 + HALF * (o.abs() + HALF * size)
                    assert torch.all((out[t, r].double() - o).abs() <= tol)
                t += 1
        assert torch.all(out[t:] == 7)
        # every page is somewhere once
        free = L.free.tolist()[:int(L.count)]
        held = [pg for b in range(N) for pg in table[b][:R.up(len(hist[b]), page)]]
        assert sorted(free + held) == list(range(L.p.num_pages))


def test_equal_inputs_give_equal_bits_on_another_stream():
    D, G, Hkv, page, budget = 128, 4, 8, 64, 12
    pages, table, seq, pos, k, v, q = attend_case(D, G, Hkv, page, 1, [3000] * 5, [2] * 5, 21)
    sel = ints(lists(seq, pos, Hkv, budget, page, 0, 5))
    p = problem(num_seqs=5, num_q_heads=G * Hkv, num_kv_heads=Hkv, page_size=page, num_pages=pages,
                max_pages_per_seq=len(table[0]), total_q_tokens=10, max_q_len=2,
                max_context_len=3000, layout=1)
    dev = [x.transpose(1, 2).contiguous().cuda() for x in (k, v)]
    qd, t, s, x = q.cuda(), ints(table), ints(seq), ints(pos)
    got = []
    for stream in (None, torch.cuda.Stream(), torch.cuda.Stream()):
        ws = torch.zeros(B.pa_selected_workspace_size(p, budget), dtype=torch.uint8, device="cuda")
        out = torch.zeros((10, G * Hkv, D), dtype=BF16, device="cuda")
        lse = torch.zeros((10, G * Hkv), device="cuda")
        torch.cuda.synchronize()
        for _ in range(3):
            B.pa_decode_selected(p, budget, qd, *dev, t, s, x, sel, ws, out, lse, stream=stream)
        torch.cuda.synchronize()
        got.append((out, lse))
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])


def test_two_loops_at_once_on_two_streams():
    """Every operator of two decode loops, each on a stream of its own, against the same loops
    one after the other."""
    def make():
        loops = [Loop(3, 8, 2, 128, 16, i, 4, 9, 700, seed=i) for i in range(2)]
        g = torch.Generator().manual_seed(9)
        data = [[torch.randn(L.fused.shape, generator=g).to(BF16).cuda() for _ in range(60)]
                for L in loops]
        return loops, data

    got = []
    for both in (False, True):
        loops, data = make()
        streams = [torch.cuda.Stream() for _ in loops] if both else [torch.cuda.current_stream()] * 2
        torch.cuda.synchronize()
        for i in range(60):
            for L, x, s in zip(loops, data, streams):
                with torch.cuda.stream(s):
                    L.fused.copy_(x[i])
                    L.ql.copy_(torch.tensor([3, 1 + i % 4, 2], dtype=torch.int32, device="cuda"))
                    L.step()
        torch.cuda.synchronize()
        for L in loops:
            no_error(L.err)
            assert B.pa_last_device_error(L.ws) == 0
        got.append([(L.out, L.lse, L.sel, L.table, L.lens) for L in loops])
    for one, two in zip(*got):
        for a, b in zip(one, two):
            assert torch.equal(a, b)


# ------------------------------------------- calls at the edge of what is allowed

def test_take_of_lengths_that_add_up_to_2_to_the_31():
    """No sequence's rows fit; the few rows that there are become padding, and nothing
    else is written."""
    B_, most = 3, 715827882                    # B_ * most = 2^31 - 2
    width = (most + 255) // 256
    p = problem(num_seqs=B_, num_q_heads=2, page_size=256, num_pages=4, max_pages_per_seq=width,
                total_q_tokens=5, max_q_len=most, max_context_len=most)
    table = torch.full((B_, width), -1, dtype=torch.int32, device="cuda")
    maps = [ints([-9] * 9) for _ in range(3)]
    ctx, left, err = ints([-9] * B_), ints([-9]), ints([0])
    B.pa_pages_take(p, ints([0] * B_), ints([most] * B_), table, ints([0, 1, 2, 3]), ints([4]),
                    ctx, *maps, left, err)
    for m, x in zip(maps, (-1, 0, -1)):
        assert m.tolist() == [x] * 5 + [-9] * 4
    assert ctx.tolist() == [0] * B_ and int(left) == 4 and int(err) == 1
    assert not (table != -1).any()


@pytest.mark.parametrize("most", [1, 3])
def test_attention_of_few_rows_among_many_of_padding(most):
    """Rows of no sequence before, between and far behind the others."""
    ctx, ql = [900, 70, 333], [most, 1, most]
    pages, table, seq, pos, k, v, q = attend_case(128, 4, 2, 16, 0, ctx, ql, 11)
    lead, gap, tail = 40, 70, 3000
    n0 = ql[0]
    seq = [-1] * lead + seq[:n0] + [-1] * gap + seq[n0:] + [-1] * tail
    pos = [0] * lead + pos[:n0] + [0] * gap + pos[n0:] + [0] * tail
    full = torch.zeros((len(seq), *q.shape[1:]), dtype=BF16)
    full[[i for i, b in enumerate(seq) if b >= 0]] = q
    sel = lists(seq, pos, 2, 9, 16, 0, 6)
    p = problem(num_seqs=3, num_q_heads=8, num_pages=pages, max_pages_per_seq=len(table[0]),
                total_q_tokens=len(seq), max_q_len=most, max_context_len=max(ctx))
    check_attend(p, 9, table, seq, pos, k, v, full, sel, repeat=2)


def test_tensors_on_the_host_are_refused():
    """Each tensor of each call in turn, before the library sees any."""
    p = problem(total_q_tokens=2, num_seqs=2)
    bf = lambda *s: torch.zeros(s, dtype=BF16, device="cuda")  # noqa: E731
    seq, pos, slots, err = ints([0, 1]), ints([3, 4]), ints([3, 20]), ints([0])
    table = ints([[0] * 8, [1] * 8])
    k, v, q = bf(8, 16, 2, 128), bf(8, 16, 2, 128), bf(2, 4, 128)
    kn, vn, out = bf(2, 2, 128), bf(2, 2, 128), bf(2, 4, 128)
    bounds = torch.zeros((8, 2, 2, 128), dtype=torch.int8, device="cuda")
    scale = torch.zeros((8, 2), device="cuda")
    sel = torch.zeros((2, 2, 1), dtype=torch.int32, device="cuda")
    steps, rope = B.pa_rope_steps(freq_of(128)).cuda(), B.PaRope(128, 0, 1.0)
    ws = torch.zeros(B.pa_selected_workspace_size(p, 1), dtype=torch.uint8, device="cuda")
    lse = torch.zeros((2, 4), device="cuda")
    stack, count = ints([2, 3, 4, 5, 6, 7, 0, 0]), ints([6])
    one = lambda: ints([0, 0])  # noqa: E731
    calls = [
        (B.pa_pages_take, (p, ints([3, 4]), ints([1, 1]), table, stack, count, one(), one(), one(),
                           one(), ints([0]), err)),
        (B.pa_pages_return, (p, ints([3, 4]), ints([3, 4]), table, stack, count, ints([0]), err)),
        (B.pa_rope_append, (p, rope, steps, q, kn, vn, pos, slots, out, k, None, v, None, err)),
        (B.pa_page_bounds, (p, k, slots, bounds, scale, err)),
        (B.pa_select_pages, (p, 1, 0, 0, q, bounds, scale, table, seq, pos, sel, err)),
        (B.pa_decode_selected, (p, 1, q, k, v, table, seq, pos, sel, ws, out, lse)),
    ]
    for f, args in calls:
        f(*args)
        for i, a in enumerate(args):
            if torch.is_tensor(a):
                with pytest.raises(ValueError):
                    f(*args[:i], a.cpu(), *args[i + 1:])
    torch.cuda.synchronize()
    no_error(err)
    # a 4-bit cache's scales
    x = problem(total_q_tokens=2, num_seqs=2, kv_dtype=B.PA_MX4)
    codes, s4 = (torch.zeros((8, 16, 2, n), dtype=torch.uint8, device="cuda") for n in (64, 4))
    args = (x, rope, steps, q, kn, vn, pos, slots, out, codes, s4, codes.clone(), s4.clone(), err)
    B.pa_rope_append(*args)
    for i in (9, 10, 11, 12):
        with pytest.raises(ValueError):
            B.pa_rope_append(*args[:i], args[i].cpu(), *args[i + 1:])
    torch.cuda.synchronize()
    no_error(err)


@pytest.mark.parametrize("Hkv,page,budget,ctx,ql", [
    (8, 16, 6, [70000, 200], [5, 155]),        # more pages than a warp looks at together
    (8, 16, 40, [70000], [5]),                 # a CTA a head
    (12, 16, 7, [5000, 60], [3, 20]), (5, 32, 9, [300, 60], [30, 20]), (9, 16, 3, [400], [2]),
    (1, 16, 300, [9000, 5000], [6, 4]), (3, 16, 70, [2000], [75]),
])
def test_attention_of_rows_of_one_sequence_by_heads(Hkv, page, budget, ctx, ql):
    """A row's heads in one CTA, or shared out among several; a warp a head, or more."""
    test_attention_of_rows_of_one_sequence(64, 2, Hkv, page, 0, 0, budget, ctx, ql, "plain", 0)
    if len(ctx) == 1:
        test_attention_of_rows_of_one_sequence(64, 2, Hkv, page, 0, 90, budget, ctx, ql, "holes", 0)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 5, 2 ** 30 + 1, 41])
@pytest.mark.parametrize("D,G,page,ctx,ql", [(128, 4, 16, [18, 35, 16], [6, 5, 6]),
                                             (64, 2, 32, [50, 17], [6, 3]),
                                             (64, 5, 16, [34], [6])])
def test_a_window_of_the_whole_context_hides_nothing(D, G, page, ctx, ql, window):
    """Windows no shorter than any context, up to the largest number there is: every bit as with
    none, rows of a sequence on both sides of a step's first key among them."""
    window = max(window, max(ctx))
    pages, table, seq, pos, k, v, q = attend_case(D, G, 2, page, 0, ctx, ql, 3)
    budget = R.up(max(ctx), page)
    sel = lists(seq, pos, 2, budget, page, 0, 5)
    kw = dict(num_seqs=len(ctx), num_q_heads=2 * G, head_dim=D, page_size=page, num_pages=pages,
              max_pages_per_seq=len(table[0]), total_q_tokens=len(seq), max_q_len=max(ql),
              max_context_len=max(ctx))
    none = check_attend(problem(**kw), budget, table, seq, pos, k, v, q, sel)
    got = check_attend(problem(window=window, **kw), budget, table, seq, pos, k, v, q, sel)
    assert torch.equal(got[0], none[0]) and torch.equal(got[1], none[1])


def test_pages_of_one_buffer():
    """Every tensor of the two calls a slice of one buffer, back to back: no overlap."""
    seq, q, page, pages, width, rows = [5, 0, 31], [12, 1, 1], 16, 9, 4, 15
    sizes = dict(seq=3, table=3 * width, ctx=3, free=pages, left=1, q=3, count=1, rs=rows, pos=rows,
                 slots=rows, err=1)
    arena, at, s = ints([-9] * sum(sizes.values())), 0, {}
    for name, n in sizes.items():
        s[name] = arena[at:at + n]
        at += n
    table = [[0, -1, -1, -1], [-1] * 4, [1, 2, -1, -1]]
    stack = [3, 4, 5, 6, 7, 8, -1, -1, -1]
    for name, x in (("seq", seq), ("q", q), ("table", sum(table, [])), ("free", stack),
                    ("count", [6]), ("err", [0])):
        s[name].copy_(ints(x))
    p = problem(num_seqs=3, page_size=page, num_pages=pages, max_pages_per_seq=width,
                total_q_tokens=rows, max_q_len=12, max_context_len=width * page)
    t = s["table"].view(3, width)
    B.pa_pages_take(p, s["seq"], s["q"], t, s["free"], s["count"], s["ctx"], s["rs"], s["pos"],
                    s["slots"], s["left"], s["err"])
    want = R.take(seq, q, table, stack, 6, page=page, pages=pages, rows=rows, max_q=12,
                  max_ctx=width * page)
    maps = list(zip(s["rs"].tolist(), s["pos"].tolist(), s["slots"].tolist()))
    assert (t.tolist(), s["ctx"].tolist(), maps, int(s["left"]), int(s["err"])) == want
    s["count"].copy_(s["left"])
    s["q"].zero_()                            # the lengths that stay
    B.pa_pages_return(p, s["ctx"], s["q"], t, s["free"], s["count"], s["left"], s["err"])
    assert int(s["left"]) == pages and sorted(s["free"].tolist()) == list(range(pages))
    no_error(s["err"])


@pytest.mark.parametrize("T,stride", [(1, 0), (1, 24), (9, 0), (9, 24)])
def test_rope_within_one_buffer(T, stride):
    """q, k_new, v_new and q_out back to back in one buffer; and the only token of a fused
    projection turned in place."""
    Hq, Hkv, D, page = 4, 2, 64, 16
    p, q, k, v, slots, kc, vc, _ = rope_case(T, Hq, Hkv, D, page, 0, B.PA_BF16, strided=False, seed=3)
    steps, rope = B.pa_rope_steps(freq_of(D)).cuda(), B.PaRope(D, 0, 1.0)
    pos, err = ints([50 + 3 * i for i in range(T)]), ints([0])
    want = torch.zeros_like(q)
    B.pa_rope_append(p, rope, steps, q, k, v, pos, slots, want, kc, None, vc, None, err)
    width = (Hq + 2 * Hkv) * D + stride
    arena = torch.zeros(T * width + T * Hq * D, dtype=BF16, device="cuda")
    fused = arena[:T * width].view(T, width)
    qs, ks, vs = (fused[:, a * D:b * D].unflatten(1, (-1, D))
                  for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    for to, x in ((qs, q), (ks, k), (vs, v)):
        to.copy_(x)
    out = arena[T * width:].view(T, Hq, D)
    k2, v2 = torch.full_like(kc, math.nan), torch.full_like(vc, math.nan)
    call = lambda o: B.pa_rope_append(p, rope, steps, qs, ks, vs, pos, slots, o, k2, None, v2,  # noqa: E731,E501
                                      None, err)
    call(out)
    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))  # noqa: E731
    assert same(out, want) and same(k2, kc) and same(v2, vc)
    if T == 1:
        call(arena[:Hq * D].view(T, Hq, D))
        assert same(arena[:Hq * D].view(T, Hq, D), want)
    no_error(err)


# ------------------------------------- rows of one sequence: errors, and non-finite values

@pytest.mark.parametrize("ctas", [0, 5, 700])
@pytest.mark.parametrize("D,G,Hkv,page,layout", [(128, 4, 2, 16, 0), (64, 5, 3, 32, 1),
                                                 (128, 11, 1, 16, 1), (64, 1, 9, 16, 0)])
def test_rows_of_one_sequence_past_bad_entries(D, G, Hkv, page, layout, ctas):
    """A row that cannot be among good ones, a unit of none but such, sequences that are none;
    entries and pages that are none, listed by one row or by several."""
    budget = 7
    pages, table, seq, pos, k, v, q = attend_case(D, G, Hkv, page, layout, [300, 200, 64],
                                                  [5, 3, 2], 9)
    sel = lists(seq, pos, Hkv, budget, page, 0, 5)
    p = problem(num_seqs=3, num_q_heads=G * Hkv, num_kv_heads=Hkv, head_dim=D, page_size=page,
                num_pages=pages, max_pages_per_seq=len(table[0]), layout=layout,
                total_q_tokens=15, max_q_len=5, max_context_len=300, num_ctas=ctas)
    q = torch.cat((q, q[:5]))
    more = dict(seq=seq + [-1] + [3, 3] + [1, 1], pos=pos + [0] + [7, 8] + [9, 10])
    sel = sel + sel[:1] + sel[8:10] + lists([1, 1], [9, 10], Hkv, budget, page, 0, 6)
    run = lambda code, s=sel, t=table, **kw: check_attend(  # noqa: E731
        p, budget, t, k=k, v=v, q=q, sel=s, code=code, repeat=2, **{**more, **kw})
    run(1)                                    # a sequence that is none
    good = dict(seq=[b if b < 3 else -1 for b in more["seq"]])
    run(0, **good)
    for bad in (300, -1, 2 ** 31 - 1, -2 ** 31):
        at = list(more["pos"])
        at[1] = bad                           # among rows 0 .. 4
        run(1, pos=at, **good)
        at = list(more["pos"])
        at[8] = at[9] = bad                   # both rows of sequence 2
        run(1, pos=at, **good)
    for entry in (pos[0] // page + 1, 2 ** 31 - 1, 2 ** 26, -2, -2 ** 31):
        s = [[list(x) for x in r] for r in sel]
        s[0][0][2] = s[6][Hkv - 1][1] = entry
        s[1][0][2] = entry                    # the same one by two rows
        run(1, s=s, **good)
    t = [list(r) for r in table]
    t[0][sel[2][0][1]], t[1][sel[5][0][0]], t[2][0] = -1, pages, 2 ** 31 - 1
    run(2, t=t, **good)
    run(0, s=[[[-1] * budget] * Hkv] * 15, **good)


@pytest.mark.parametrize("ctas", [0, 5, 700])
@pytest.mark.parametrize("D,G,page,rows", [(128, 4, 16, 4), (64, 3, 32, 6), (128, 16, 16, 2),
                                           (64, 8, 16, 4)])
def test_non_finite_values_in_units_that_are_split(D, G, page, rows, ctas):
    """An infinity or NaN of K or V in a page that one row of several lists, in lists long enough
    for several CTAs: the others' results are right, and its own column (V) or row (a NaN in K)
    is not finite."""
    ctx = 2600
    pages, table, seq, pos, k, v, q = attend_case(D, G, 1, page, 0, [ctx], [rows], 9)
    n = R.up(ctx, page)
    budget = n // 2
    g = torch.Generator().manual_seed(4)
    # (the first pages of all but the last row's list are common to the others', one is its own)
    own = n - 9
    rest = [s for s in range(n - 5) if s != own]
    sel = []
    for r in range(rows):
        pick = [rest[i] for i in torch.randperm(len(rest), generator=g)[:budget - 1].tolist()]
        sel.append([sorted(pick + [own if r == 1 else n - 7 if n - 7 not in pick else n - 5])])
    p = problem(num_q_heads=G, num_kv_heads=1, head_dim=D, page_size=page, num_pages=pages,
                max_pages_per_seq=n, total_q_tokens=rows, max_q_len=rows, max_context_len=ctx,
                num_ctas=ctas)
    ws = torch.zeros(B.pa_selected_workspace_size(p, budget), dtype=torch.uint8, device="cuda")
    check_attend(p, budget, table, seq, pos, k, v, q, sel)
    for value in (math.inf, -math.inf, math.nan):
        for which in "kv":
            k2, v2 = k.clone(), v.clone()
            (k2 if which == "k" else v2)[table[0][own], 3, 0, 7] = value
            out = torch.zeros((rows, G, D), dtype=BF16, device="cuda")
            lse = torch.zeros((rows, G), device="cuda")
            B.pa_decode_selected(p, budget, q.cuda(), k2.cuda(), v2.cuda(), ints(table), ints(seq),
                                 ints(pos), ints(sel), ws, out, lse)
            assert B.pa_last_device_error(ws) == 0
            for r in range(rows):
                if r == 1:
                    continue
                at = [x for s in sel[r][0] for x in range(s * page, s * page + page)]
                kk, vv = (torch.cat([x[table[0][s], :, 0] for s in sel[r][0]]) for x in (k, v))
                o, L, size, big = R.attend(q[r], kk, vv, at, pos[r], 0, p.sm_scale)
                ds = (D + 16) * 2.0 ** -24 * big[:, None] + 2.0 ** -20
                tol = (HALF + 2 * ds) * size * 1.01 + HALF * (o.abs() + HALF * size)
                assert torch.all((out[r].cpu().double() - o).abs() <= tol), (value, which, r)
                far = (lse[r].cpu().double() - L).abs()
                assert torch.all(far <= ds[:, 0] + 2.0 ** -22 * (1 + L.abs()))
            if which == "v":
                bad = ~torch.isfinite(out[1])
                assert bad[:, 7].all() and not bad[:, :7].any() and not bad[:, 8:].any()
                assert torch.isfinite(lse[1]).all()
            elif value != value:
                assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()


@pytest.mark.parametrize("Hq,Hkv,D,page,layout", [(8, 2, 128, 16, 0), (6, 3, 64, 32, 1)])
def test_a_step_with_a_sequence_that_gets_no_pages(Hq, Hkv, D, page, layout):
    """Its rows become padding in the middle of the step's; the others' results are those of a
    step without it."""
    def two_steps(ql):
        L = Loop(3, Hq, Hkv, D, page, layout, 3, 40, 4 * page, seed=2)
        g = torch.Generator().manual_seed(4)
        L.fused.copy_(torch.randn(L.fused.shape, generator=g).to(BF16))
        L.ql.copy_(ints([5, page, 3]))
        L.step()
        no_error(L.err)
        L.count.fill_(0)                      # somebody else has the rest of the pool
        new = torch.randn((3, 2, L.fused.shape[1]), generator=g).to(BF16).cuda()
        L.fused[:sum(ql)].copy_(torch.cat([new[b, :n] for b, n in enumerate(ql)]))
        L.ql.copy_(ints(ql))
        for x, fill in ((L.out, 7.0), (L.lse, 7.0), (L.qr, 7.0), (L.sel, -9)):
            x.fill_(fill)
        L.step()
        return L

    a, b = two_steps([1, 2, 2]), two_steps([1, 0, 2])
    assert int(a.err) == B.PA_DEV_NO_PAGES and int(b.err) == 0
    assert B.pa_last_device_error(a.ws) == 0
    assert a.seq.tolist() == [0, -1, -1, 2, 2] + [-1] * 35
    assert a.lens.tolist() == b.lens.tolist() == [6, page, 5]
    for x, y, fill in ((a.out, b.out, 7.0), (a.lse, b.lse, 7.0), (a.qr, b.qr, 7.0),
                       (a.sel, b.sel, -9)):
        assert torch.equal(x[[0, 3, 4]], y[:3]) and torch.isfinite(x[:5].float()).all()
        assert torch.all(x[1:3] == fill) and torch.all(x[5:] == fill)
    for x, y in ((a.k, b.k), (a.v, b.v), (a.sc, b.sc), (a.bnd, b.bnd)):
        assert torch.equal(x.view(torch.int8), y.view(torch.int8))


def test_selection_with_the_largest_budget_there_is():
    """All pages, and -1 behind them up to entry 2^31 - 2; nothing behind that."""
    budget, pos, page = 2 ** 31 - 1, 100, 16
    p = problem(num_q_heads=1, num_kv_heads=1, head_dim=64, page_size=page)
    sel = torch.full((budget + 33,), -7, dtype=torch.int32, device="cuda")
    bnd, sc = torch.zeros((8, 1, 2, 64), dtype=torch.int8).cuda(), torch.ones((8, 1)).cuda()
    err = ints([0])
    B.pa_select_pages(p, budget, 0, 0, torch.zeros((1, 1, 64), dtype=BF16, device="cuda"), bnd, sc,
                      ints([list(range(8))]), ints([0]), ints([pos]), sel, err)
    no_error(err)
    assert sel[:7].tolist() == list(range(7))
    assert int(sel[7:budget].max()) == -1 == int(sel[7:budget].min())
    assert sel[budget:].tolist() == [-7] * 33
