"""The cache operators (include/pa_cache.h) against their 64-bit plain forms.

Tolerances follow the arithmetic.  Unit roundoffs: bf16 2^-8, f16 2^-11, fp32
2^-24.  Writing, reading back and evicting move or round exactly representable
values: equal bits.  Decode rounds each probability to f16 (2^-11 of sum p |v|)
and the result to bf16; its scores carry the fp32 sum of D products.  Key
weights carry the same score error through the exponential.
"""
import math

import pytest
import torch

from paged_attention_gb300 import binding as B

import cache_ref as R

pytestmark = pytest.mark.gpu

NHD, HND, BF16, MX4 = R.NHD, R.HND, R.BF16, R.MX4


def dev(t):
    return None if t is None else t.cuda()


def error_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def same(a, b):
    """Equal values, NaN equal to NaN."""
    a, b = a.cpu().double(), b.cpu().double()
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


# -------------------------------------------------------------------- write

def append(case, new_k, new_v, ctx=None, ql=None, weights=None, **kw):
    (k, ks), (v, vs) = case.empty(), case.empty()
    k, ks, v, vs = dev(k), dev(ks), dev(v), dev(vs)
    c, q = case.lens()
    err = error_word()
    B.pa_kv_append(case.problem(B, **kw), new_k, new_v, dev(case.table),
                   c if ctx is None else ctx, q if ql is None else ql, k, ks, v, vs, weights, err)
    torch.cuda.synchronize()
    return k, ks, v, vs, int(err.item())


def new_rows(case, dense):
    return torch.cat([d[c - q:] for d, c, q in zip(dense, case.ctx, case.ql)])


@pytest.mark.parametrize("kv", [BF16, MX4])
@pytest.mark.parametrize("dim,kv_heads,page,layout", [
    (128, 2, 16, NHD), (64, 1, 32, HND), (64, 3, 16, NHD), (128, 5, 64, HND)])
@pytest.mark.parametrize("ctx,ql", [
    ([1], [1]), ([37, 16, 100], [37, 0, 3]), ([33] * 40, [1] * 40), ([260, 5], [130, 5])])
def test_append_writes_the_new_rows_and_nothing_else(kv, dim, kv_heads, page, layout, ctx, ql):
    case = R.Case(ctx, ql, heads=kv_heads, kv_heads=kv_heads, dim=dim, page=page, layout=layout,
                  kv=kv, seed=3)
    want = [case.empty(), case.empty()]
    for b, (c, q) in enumerate(zip(ctx, ql)):
        for (cache, scales), dense in zip(want, (case.kd[b], case.vd[b])):
            rows, pos = dense[c - q:], range(c - q, c)
            if kv == BF16:
                case.put(cache, b, pos, rows)
            else:
                codes, sc = R.quantise(rows)
                case.put(cache, b, pos, codes)
                case.put(scales, b, pos, sc)
    k, ks, v, vs, err = append(case, new_rows(case, case.kd).cuda(), new_rows(case, case.vd).cuda())
    assert err == 0
    assert same(k, want[0][0]) and same(v, want[1][0])
    if kv == MX4:
        assert same(ks, want[0][1]) and same(vs, want[1][1])


def test_append_takes_slices_of_a_fused_projection_and_clears_weights():
    case = R.Case([50, 9], [4, 9], heads=8, kv_heads=2, dim=64, page=16, seed=5)
    width = (8 + 4) * 64
    fused = torch.randn((13, width)).to(torch.bfloat16).cuda()
    k_new = fused[:, 512:640].unflatten(1, (2, 64))
    v_new = fused[:, 640:].unflatten(1, (2, 64))
    w = torch.full((case.num_pages, 2, 16), 7.0, device="cuda")
    got = append(case, k_new, v_new, weights=w)
    dense = append(case, k_new.contiguous(), v_new.contiguous())
    for a, b in zip(got[:4], dense[:4]):
        assert torch.equal(a, b)
    want = torch.full((case.num_pages, 2, 16), 7.0)
    for b, (c, q) in enumerate(zip(case.ctx, case.ql)):
        for p in range(c - q, c):
            want[int(case.table[b, p // 16]), :, p % 16] = 0
    assert same(w, want)


def test_quantisation_edges_and_read_back():
    """Every tie, saturation, subnormals, the largest bf16, zeros, infinities
    and NaN: the codes are the plain form's, and reading back gives the values
    they stand for."""
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.5, 6.0, 7.5, 0.0, -0.0, -0.25, -5.0, 0.3, 4.0]
    rows = []
    for e in (-140, -133, -130, -128, -127, -126, -125, -124, -20, 0, 1, 100, 120, 124, 125):
        rows.append([t * 2.0 ** e for t in ties] * 8)
    rows.append([0.0] * 128)
    rows.append([3.3895e38] + [1.0] * 127)
    for bad in (math.inf, -math.inf, math.nan):
        rows.append([1.0] * 40 + [bad] + [2.0] * 87)
    x = torch.tensor(rows, dtype=torch.float64).to(torch.bfloat16)[:, None].contiguous()
    n = x.shape[0]
    case = R.Case([n], [n], heads=1, kv_heads=1, dim=128, page=16, seed=1)
    k, ks, v, vs, err = append(case, x.cuda(), x.flip(0).contiguous().cuda())
    assert err == 0
    codes, sc = R.quantise(x)
    assert same(case.get(k.cpu(), 0, n), codes) and same(case.get(ks.cpu(), 0, n), sc)
    out = [torch.zeros(case.shape(128), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    c, q = case.lens()
    e = error_word()
    B.pa_kv_expand(case.problem(B), k, ks, v, vs, dev(case.table), c, q, dev(case.table),
                   case.num_pages, out[0], out[1], e)
    torch.cuda.synchronize()
    assert int(e.item()) == 0
    want = R.dequantise(codes, sc)
    assert same(case.get(out[0].cpu(), 0, n), want.to(torch.bfloat16))
    assert same(case.get(out[1].cpu(), 0, n), want.flip(0).to(torch.bfloat16))


@pytest.mark.parametrize("dim,page,layout", [(128, 16, HND), (64, 32, NHD)])
def test_expand_reads_the_last_tokens_into_other_pages(dim, page, layout):
    ctx, ql = [70, 33, 1, 20], [70, 5, 1, 0]
    case = R.Case(ctx, ql, heads=3, kv_heads=3, dim=dim, page=page, layout=layout, seed=2)
    pages = 40
    dst = torch.full((4, case.mpps + 2), -1, dtype=torch.int32)
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(9))
    at = 0
    for b, c in enumerate(ctx):
        n = -(-c // page)
        dst[b, :n] = perm[at:at + n].int()
        at += n
    shape = (pages,) + case.shape(dim)[1:]
    out = [torch.full(shape, 5.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    want = [torch.full(shape, 5.0, dtype=torch.bfloat16) for _ in "kv"]
    for b, (c, q) in enumerate(zip(ctx, ql)):
        for w, n in zip(want, "kv"):
            case.put(w, b, range(c - q, c), case.rows(n, b)[c - q:].to(torch.bfloat16), dst)
    c, q = case.lens()
    err = error_word()
    B.pa_kv_expand(case.problem(B), dev(case.k), dev(case.ks), dev(case.v), dev(case.vs),
                   dev(case.table), c, q, dev(dst), pages, out[0], out[1], err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert same(out[0], want[0]) and same(out[1], want[1])


@pytest.mark.parametrize("layout", [NHD, HND])
@pytest.mark.parametrize("dim,kv_heads", [(128, 9), (128, 20), (64, 33), (128, 7)])
def test_tokens_wider_and_narrower_than_a_cta(dim, kv_heads, layout):
    """K and V of a token are 2 * kv_heads * dim / 8 threads' work: more than
    one CTA's, with a remainder, or fewer than it has."""
    ctx, ql = [45, 18, 3], [45, 1, 2]
    case = R.Case(ctx, ql, heads=kv_heads, kv_heads=kv_heads, dim=dim, page=16, layout=layout, seed=6)
    fresh = R.Case(ctx, ql, heads=kv_heads, kv_heads=kv_heads, dim=dim, page=16, layout=layout, seed=6)
    w = torch.full((case.num_pages, kv_heads, 16), 3.0, device="cuda")
    k, ks, v, vs, err = append(fresh, new_rows(case, case.kd).cuda(), new_rows(case, case.vd).cuda(),
                               weights=w)
    assert err == 0
    want_w = torch.full((case.num_pages, kv_heads, 16), 3.0)
    for b, (c, q) in enumerate(zip(ctx, ql)):
        for got, sc, full, full_sc in ((k, ks, case.k, case.ks), (v, vs, case.v, case.vs)):
            assert same(case.get(got.cpu(), b, c)[c - q:], case.get(full, b, c)[c - q:])
            assert same(case.get(sc.cpu(), b, c)[c - q:], case.get(full_sc, b, c)[c - q:])
        for p in range(c - q, c):
            want_w[int(case.table[b, p // 16]), :, p % 16] = 0
    assert same(w, want_w)
    shape = case.shape(dim)
    out = [torch.full(shape, 5.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    cl, qq = case.lens()
    err = error_word()
    B.pa_kv_expand(case.problem(B), k, ks, v, vs, dev(case.table), cl, qq, dev(case.table),
                   case.num_pages, out[0], out[1], err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for b, (c, q) in enumerate(zip(ctx, ql)):
        for got, n in zip(out, "kv"):
            want = case.rows(n, b)[c - q:].to(torch.bfloat16)
            assert same(case.get(got.cpu(), b, c)[c - q:], want)
            assert bool((case.get(got.cpu(), b, c)[:c - q] == 5.0).all())


def test_more_tokens_than_one_wave_holds():
    """70001 tokens of one head: rows i of the new tokens hold the number i."""
    n, page = 70001, 256
    pages = -(-n // page)
    rows = torch.arange(n, dtype=torch.int32).view(n, 1, 1).expand(n, 1, 32)
    x = rows.contiguous().view(torch.int16).view(torch.bfloat16).cuda()      # [n, 1, 64], any bits
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(3)).int().cuda().view(1, -1)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    p = B.PaProblem(num_seqs=1, num_q_heads=1, num_kv_heads=1, head_dim=64, page_size=page,
                    num_pages=pages, max_pages_per_seq=pages, total_q_tokens=n, max_q_len=n,
                    max_context_len=n, kv_dtype=BF16, sm_scale=1.0)
    k, v = (torch.zeros((pages, page, 1, 64), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    err = error_word()
    B.pa_kv_append(p, x, x, table, lens, lens, k, None, v, None, None, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for cache in (k, v):
        got = cache.view(torch.int16)[table[0].long()].reshape(-1, 64)[:n].contiguous()
        assert torch.equal(got, x.view(torch.int16).view(n, 64))


def test_write_skips_what_it_cannot_place():
    """A page outside the pool, lengths that contradict each other, q_lens that
    do not add up: flagged, the rows concerned left out, the others written."""
    case = R.Case([40, 20, 10], [2, 2, 2], heads=1, kv_heads=1, dim=64, page=16, seed=4)
    x = torch.randn((6, 1, 64)).to(torch.bfloat16).cuda()
    case.table[1, 1] = case.num_pages            # tokens 18, 19 of sequence 1
    k, ks, v, vs, err = append(case, x, x)
    assert err == B.PA_DEV_BAD_PAGE
    good, _ = R.quantise(x[:2].cpu())
    assert same(case.get(k.cpu(), 0, 40)[38:], good)
    assert same(case.get(k.cpu(), 2, 10)[8:], R.quantise(x[4:].cpu())[0])
    case.table[1, 1] = -1
    assert append(case, x, x)[-1] == B.PA_DEV_BAD_PAGE
    case = R.Case([40, 20, 10], [2, 2, 2], heads=1, kv_heads=1, dim=64, page=16, seed=4)
    ctx = torch.tensor([40, 1, 10], dtype=torch.int32, device="cuda")      # 2 new of 1
    k, ks, v, vs, err = append(case, x, x, ctx=ctx)
    assert err == B.PA_DEV_BAD_LENGTHS
    assert same(case.get(k.cpu(), 2, 10)[8:], R.quantise(x[4:].cpu())[0])
    ql = torch.tensor([2, 2, 1], dtype=torch.int32, device="cuda")         # 5 of 6 rows
    assert append(case, x, x, ql=ql)[-1] == B.PA_DEV_BAD_LENGTHS
    ql = torch.tensor([2, 2, -1], dtype=torch.int32, device="cuda")
    assert append(case, x, x, ql=ql)[-1] == B.PA_DEV_BAD_LENGTHS


# ------------------------------------------------------------------- decode

def decode(case, num_ctas=0, stream=None, **kw):
    p = case.problem(B, num_ctas=num_ctas, **kw)
    n = B.pa_mx4_workspace_size(p)
    assert n > 0
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    out = torch.full((case.total_q, case.heads, case.dim), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((case.total_q, case.heads), 9.0, device="cuda")
    c, q = case.lens()
    B.pa_decode_mx4(p, case.q.cuda(), dev(case.k), dev(case.ks), dev(case.v), dev(case.vs),
                    dev(case.table), c, q, ws, out, lse, stream)
    torch.cuda.synchronize()
    return out, lse, ws


def check_decode(case, **kw):
    out, lse, ws = decode(case, **kw)
    assert B.pa_last_device_error(ws) == 0
    ref, rl, mag, big = R.attention(case)
    score = (case.dim + 8) * 2.0 ** -24 * big
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2.0 ** -14 + 2 * score[..., None]) * mag + 1e-30
    d = (out.cpu().double() - ref).abs()
    assert bool((d <= tol).all()), f"out off by {float((d / tol).max())} of its tolerance"
    tl = score + 2.0 ** -20 + rl.abs() * 2.0 ** -21
    dl = (lse.cpu().double() - rl).abs()
    assert bool((dl <= tl).all()), f"lse off by {float((dl / tl).max())} of its tolerance"
    return out, lse


@pytest.mark.parametrize("layout", [NHD, HND])
@pytest.mark.parametrize("dim,heads,kv_heads,page,ctx,ql", [
    (128, 4, 2, 16, [1], [1]),
    (128, 1, 1, 16, [31, 32, 33, 64, 65], [1, 1, 1, 1, 1]),
    (128, 4, 1, 64, [200, 1, 0, 63], [2, 1, 0, 0]),
    (128, 16, 2, 16, [129, 700], [1, 1]),
    (128, 16, 2, 32, [129, 700], [2, 1]),
    (128, 24, 3, 128, [90, 3], [3, 3]),
    (128, 16, 1, 16, [300], [2]),
    (128, 5, 1, 256, [513, 2], [6, 2]),
    (64, 4, 1, 16, [37, 100, 80], [1, 1, 4]),
    (64, 3, 3, 16, [37, 101], [1, 3]),
    (64, 16, 1, 32, [70, 1], [2, 1]),
    (64, 16, 2, 16, [260, 64], [4, 2]),
    (64, 64, 1, 64, [150], [1]),
])
def test_decode_against_the_plain_form(layout, dim, heads, kv_heads, page, ctx, ql):
    check_decode(R.Case(ctx, ql, heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                        layout=layout, seed=11))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window", [1, 7, 32, 100, 5000])
def test_decode_window(dim, window):
    check_decode(R.Case([300, 40, 9], [3, 1, 2], heads=4, kv_heads=2, dim=dim, window=window,
                        seed=12))


@pytest.mark.parametrize("num_ctas", [1, 2, 5, 64, 152, 1024])
def test_decode_split_over_any_number_of_ctas(num_ctas):
    """The same work cut in other places: equal up to rounding, each within tolerance."""
    case = R.Case([1500, 3, 640, 64], [1, 2, 1, 0], heads=4, kv_heads=2, dim=128, seed=13)
    check_decode(case, num_ctas=num_ctas)
    check_decode(case, num_ctas=num_ctas, unit_cost=-1)


@pytest.mark.parametrize("dim,heads,kv_heads,ctx,ql,window", [
    (64, 16, 2, [500, 8, 70, 333, 90], [8, 1, 4, 5, 0], 0),      # 64, 8, 32, 40 and no rows
    (64, 11, 1, [1200, 40], [5, 3], 0),                          # 55 and 33 rows of 11 heads
    (64, 64, 1, [2500, 1], [1, 1], 0),                           # one token of 64 heads, split
    (64, 6, 1, [300, 299], [9, 10], 40),                         # 54 and 60 rows, a window
    (128, 16, 2, [500, 8, 70, 333, 90], [4, 1, 2, 3, 0], 0),     # 32, 8, 16, 24 and no rows
    (128, 9, 1, [1200, 40], [3, 2], 0),                          # 27 and 18 rows of 9 heads
    (128, 32, 1, [2500, 1], [1, 1], 30),
])
def test_decode_of_two_blocks_of_rows(dim, heads, kv_heads, ctx, ql, window):
    check_decode(R.Case(ctx, ql, heads=heads, kv_heads=kv_heads, dim=dim, page=16, window=window,
                        seed=71))


def test_decode_many_short_sequences():
    g = torch.Generator().manual_seed(8)
    ctx = torch.randint(1, 90, (150,), generator=g).tolist()
    ql = [min(c, i % 3) for i, c in enumerate(ctx)]
    check_decode(R.Case(ctx, ql, heads=2, kv_heads=1, dim=64, seed=14))


def test_decode_values_of_very_different_size():
    """Keys and values over many powers of two: scores far apart, V's scales
    rising late and falling again."""
    case = R.Case([200, 170], [1, 2], heads=4, kv_heads=2, dim=128, seed=15)
    f = torch.exp2(torch.linspace(-12, 6, 200))[:, None, None]
    case.vd[0] = (case.vd[0].float() * f).to(torch.bfloat16)
    case.vd[1] = (case.vd[1].float() * f.flip(0)[:170]).to(torch.bfloat16)
    case.kd[0] = (case.kd[0].float() * torch.exp2(torch.arange(200) % 7 - 4.0)[:, None, None]).to(torch.bfloat16)
    case.fill()
    check_decode(case)
    # queries near the ends of bf16's range, keys to match
    case = R.Case([70], [2], heads=2, kv_heads=1, dim=64, seed=16, kmag=2.0 ** -100)
    case.q = (case.q.float() * 2.0 ** 98).to(torch.bfloat16)
    check_decode(case)
    case = R.Case([70], [2], heads=2, kv_heads=1, dim=64, seed=16, kmag=2.0 ** 98)
    case.q = (case.q.float() * 2.0 ** -100).to(torch.bfloat16)
    check_decode(case)


def test_decode_nan_reaches_only_the_rows_that_see_it():
    case = R.Case([100, 90], [3, 2], heads=4, kv_heads=2, dim=128, seed=17, window=60)
    # a hidden value: the last key of sequence 0, seen by its last query alone
    for cache, col in ((case.vs, 2), (case.ks, 1)):
        c2 = R.Case([100, 90], [3, 2], heads=4, kv_heads=2, dim=128, seed=17, window=60)
        target = c2.vs if cache is case.vs else c2.ks
        pg, s = int(c2.table[0, 99 // 16]), 99 % 16
        target[pg, s, 1, col] = 255                       # KV head 1, one block
        pg, s = int(c2.table[1, 0]), 3                    # before every window
        target[pg, s, 0, col] = 255
        out, lse, _ = decode(c2)
        clean, clean_lse, _ = decode(case)
        ref = R.attention(c2)
        nan = torch.isnan(ref[0])
        assert torch.equal(torch.isnan(out.cpu().float()), nan)
        assert bool(nan.any()) and torch.equal(torch.isnan(lse.cpu()), torch.isnan(ref[1]))
        # rows that do not see it keep their bits
        rows = ~nan.any(-1)
        assert torch.equal(out.cpu()[rows], clean.cpu()[rows])
        assert torch.equal(lse.cpu()[rows], clean_lse.cpu()[rows])


def test_decode_is_deterministic_without_splits_and_leaves_other_rows():
    case = R.Case([300, 20, 77], [1, 0, 2], heads=4, kv_heads=2, dim=128, seed=18)
    a, al, _ = decode(case)
    b, bl, _ = decode(case)
    assert torch.equal(a, b) and torch.equal(al, bl)
    # lse may be left out
    p = case.problem(B)
    ws = torch.zeros(B.pa_mx4_workspace_size(p), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(a)
    c, q = case.lens()
    B.pa_decode_mx4(p, case.q.cuda(), dev(case.k), dev(case.ks), dev(case.v), dev(case.vs),
                    dev(case.table), c, q, ws, out, None)
    torch.cuda.synchronize()
    assert torch.equal(out, a)


def test_one_workspace_serves_problem_after_problem():
    """Calls of different problems, split over many CTAs, in one workspace, and
    two streams with a workspace each: bit for bit what a fresh one gives."""
    cases = [R.Case([900, 5, 300], [1, 1, 1], heads=4, kv_heads=2, dim=64, seed=51),
             R.Case([40] * 30, [1] * 30, heads=3, kv_heads=1, dim=128, seed=52),
             R.Case([1500], [3], heads=8, kv_heads=1, dim=128, seed=53)]
    calls = []
    for c in cases:
        p = c.problem(B)
        calls.append((p, c.q.cuda(), dev(c.k), dev(c.ks), dev(c.v), dev(c.vs), dev(c.table),
                      *c.lens()))
    size = max(B.pa_mx4_workspace_size(a[0]) for a in calls)

    def run(a, ws, stream=None):
        out = torch.full((a[1].shape[0], a[1].shape[1], a[1].shape[2]), 7.0, dtype=torch.bfloat16,
                         device="cuda")
        lse = torch.full(out.shape[:2], 7.0, device="cuda")
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        B.pa_decode_mx4(a[0], *a[1:], ws, out, lse, stream)
        return out, lse

    fresh = [run(a, torch.zeros(size, dtype=torch.uint8, device="cuda")) for a in calls]
    torch.cuda.synchronize()
    spaces = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(24):
        got.append((i % 3, run(calls[i % 3], spaces[i % 2], streams[i % 2])))
    torch.cuda.synchronize()
    for i, (out, lse) in got:
        assert torch.equal(out, fresh[i][0]) and torch.equal(lse, fresh[i][1])
    for ws in spaces:
        assert B.pa_last_device_error(ws) == 0


def test_decode_flags_bad_pages_and_lengths():
    case = R.Case([100, 50], [1, 1], heads=2, kv_heads=1, dim=64, seed=19)
    clean, _, _ = decode(case)
    case.table[0, 2] = case.num_pages + 5
    out, lse, ws = decode(case)
    assert B.pa_last_device_error(ws) == B.PA_DEV_BAD_PAGE
    assert torch.equal(out[1], clean[1])
    case = R.Case([100, 50], [1, 1], heads=2, kv_heads=1, dim=64, seed=19)
    case.ctx[0] = 0                                   # q_len 1 of no tokens
    out, lse, ws = decode(case, max_context_len=100)
    assert B.pa_last_device_error(ws) == B.PA_DEV_BAD_LENGTHS
    assert torch.equal(out[1], clean[1])
    # q_lens that run past the rows there are: the rows that exist are computed
    case = R.Case([100, 50], [1, 1], heads=2, kv_heads=1, dim=64, seed=19)
    ql = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    p = case.problem(B, max_q_len=2)
    ws = torch.zeros(B.pa_mx4_workspace_size(p), dtype=torch.uint8, device="cuda")
    out = torch.full((2, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    B.pa_decode_mx4(p, case.q.cuda(), dev(case.k), dev(case.ks), dev(case.v), dev(case.vs),
                    dev(case.table), case.lens()[0], ql, ws, out, None)
    torch.cuda.synchronize()
    assert B.pa_last_device_error(ws) == B.PA_DEV_BAD_LENGTHS
    assert torch.equal(out[0], clean[0]) and bool((out[1] == 9.0).all())


# ------------------------------------------------------------------ weights

def run_weights(case, lse, start, **kw):
    w = start.clone().cuda()
    c, q = case.lens()
    err = error_word()
    B.pa_key_weights(case.problem(B, **kw), case.q.cuda(), dev(case.k), dev(case.ks),
                     dev(case.table), c, q, lse.float().cuda(), w, err)
    torch.cuda.synchronize()
    return w.cpu().double(), int(err.item())


def check_weights(case, lse=None):
    if lse is None:
        lse = R.attention(case)[1].float().double()
    g = torch.Generator().manual_seed(1)
    start = torch.rand((case.num_pages, case.kv_heads, case.page), generator=g)
    got, err = run_weights(case, lse, start)
    assert err == 0
    add, tol = R.key_weights(case, lse)
    want, limit = start.double().clone(), torch.zeros_like(start).double()
    for b, c in enumerate(case.ctx):
        for p in range(c):
            pg, s = int(case.table[b, p // case.page]), p % case.page
            want[pg, :, s] += add[b][:, p]
            limit[pg, :, s] = tol[b][:, p] + want[pg, :, s] * 2.0 ** -24
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    d, limit = (got - want).abs()[~nan], limit[~nan]
    assert bool((d <= limit).all()), f"off by {float((d / limit.clamp(min=1e-300)).max())}"
    again, _ = run_weights(case, lse, start)
    assert same(again, got)


@pytest.mark.parametrize("kv", [BF16, MX4])
@pytest.mark.parametrize("layout,dim,heads,kv_heads,page,ctx,ql,window", [
    (NHD, 128, 4, 2, 16, [1], [1], 0),
    (HND, 128, 4, 1, 64, [300, 1, 0, 63], [1, 1, 0, 0], 0),
    (NHD, 64, 3, 3, 16, [37, 101, 31], [1, 3, 31], 0),
    (HND, 64, 16, 2, 32, [260, 64], [40, 2], 0),
    (NHD, 128, 5, 1, 16, [600], [33], 0),
    (NHD, 64, 2, 1, 16, [300, 40], [3, 1], 25),
    (HND, 128, 4, 4, 128, [520], [140], 300),
])
def test_weights_against_the_plain_form(kv, layout, dim, heads, kv_heads, page, ctx, ql, window):
    check_weights(R.Case(ctx, ql, heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                         layout=layout, kv=kv, window=window, seed=21))


@pytest.mark.parametrize("kv", [BF16, MX4])
def test_weights_of_queries_that_see_nothing_and_of_nan_keys(kv):
    case = R.Case([80, 30], [3, 1], heads=4, kv_heads=2, dim=64, kv=kv, seed=22)
    lse = R.attention(case)[1].float().double()
    lse[1, 2] = -math.inf
    check_weights(case, lse)
    pg, s = int(case.table[0, 79 // 16]), 79 % 16    # the last key: seen by one query
    if kv == BF16:
        case.k[pg, s, 1, 5] = math.nan
    else:
        case.ks[pg, s, 1, 0] = 255
    check_weights(case, lse)


def test_weights_many_sequences_and_bad_input():
    g = torch.Generator().manual_seed(8)
    ctx = torch.randint(1, 60, (70,), generator=g).tolist()
    case = R.Case(ctx, [min(c, i % 3) for i, c in enumerate(ctx)], heads=2, kv_heads=1, dim=64,
                  kv=BF16, seed=23)
    check_weights(case)
    lse = R.attention(case)[1].float().double()
    zero = torch.zeros((case.num_pages, 1, 16))
    good, _ = run_weights(case, lse, zero)
    b = next(i for i in range(70) if case.ql[i] and case.ctx[i] > 20)
    page = int(case.table[b, 0])
    case.table[b, 0] = -7
    got, err = run_weights(case, lse, zero)
    assert err == B.PA_DEV_BAD_PAGE
    good[page] = 0
    assert same(got, good)


@pytest.mark.parametrize("kv", [BF16, MX4])
def test_weights_of_many_rows_that_see_nothing_and_of_nan_keys(kv):
    """As above with 36 and 200 query rows a head (lengths that differ, one
    without queries), and a bad page."""
    case = R.Case([80, 300, 41, 700], [9, 50, 0, 17], heads=8, kv_heads=2, dim=128, kv=kv, seed=24)
    lse = R.attention(case)[1].float().double()
    lse[1, 2] = -math.inf
    lse[20] = -math.inf
    check_weights(case, lse)
    for b, key in ((0, 79), (1, 299), (3, 690)):     # seen by the last queries only
        pg, s = int(case.table[b, key // case.page]), key % case.page
        if kv == BF16:
            case.k[pg, s, 1, 5] = math.nan
        else:
            case.ks[pg, s, 1, 0] = 255
    check_weights(case, lse)
    zero = torch.zeros((case.num_pages, 2, case.page))
    good, err = run_weights(case, lse, zero)
    assert err == 0
    page = int(case.table[3, 2])
    case.table[3, 2] = case.num_pages
    got, err = run_weights(case, lse, zero)
    assert err == B.PA_DEV_BAD_PAGE
    good[page] = 0
    assert same(got, good)


@pytest.mark.parametrize("kv,dim,heads,kv_heads,page,ctx,ql,window", [
    (BF16, 128, 7, 1, 32, [1000, 5, 513], [300, 5, 129], 0),      # all chunks, partly masked
    (MX4, 64, 6, 3, 16, [900, 257], [200, 257], 100),             # a window shorter than the tile
    (BF16, 64, 2, 2, 64, [2000], [700], 33),
    (MX4, 128, 16, 1, 256, [256, 1024], [256, 8], 0),
    (MX4, 128, 4, 2, 16, [130] * 200, [20] * 200, 0),             # more items than CTAs
    (BF16, 128, 33, 1, 16, [1, 300, 1], [1, 1, 1], 0),            # one token, 33 heads
])
def test_weights_of_many_rows(kv, dim, heads, kv_heads, page, ctx, ql, window):
    check_weights(R.Case(ctx, ql, heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                         kv=kv, window=window, seed=25))


@pytest.mark.parametrize("kv", [BF16, MX4])
@pytest.mark.parametrize("skip", [0, 2])
def test_a_weights_wait_that_runs_out_is_reported_and_the_next_call_is_clean(kv, skip):
    """One CTA's producer leaves a tile unannounced and the waits last 20 ms:
    the call ends with the error word set, the next one is a normal one."""
    # (items for more than three tiles of CTA 0, on any number of SMs)
    case = R.Case([4000], [20], heads=64, kv_heads=32, dim=64, kv=kv, page=256, seed=26)
    lse = torch.full((20, 64), 9.0).double()
    zero = torch.zeros((case.num_pages, 32, 256))
    good, err = run_weights(case, lse, zero)
    assert err == 0
    B.pa_test_inject_wait_timeout(skip, 20_000_000)
    _, err = run_weights(case, lse, zero)
    assert err == B.PA_DEV_WAIT_TIMEOUT
    again, err = run_weights(case, lse, zero)
    assert err == 0 and same(again, good)


# -------------------------------------------------------------------- evict

def run_evict(case, w, budget, first, recent, dst, **kw):
    k, ks, v, vs = dev(case.k.clone()), dev(case.ks), dev(case.v.clone()), dev(case.vs)
    ks, vs = (None, None) if ks is None else (ks.clone(), vs.clone())
    w = w.clone().cuda()
    kept = torch.full((len(case.ctx), case.kv_heads, budget), -1, dtype=torch.int32, device="cuda")
    new = torch.full((len(case.ctx),), -1, dtype=torch.int32, device="cuda")
    err = error_word()
    B.pa_kv_evict(case.problem(B, **kw), budget, first, recent, k, ks, v, vs, w, dev(case.table),
                  dev(dst), case.lens()[0], kept, new, err)
    torch.cuda.synchronize()
    return dict(k=k, ks=ks, v=v, vs=vs, w=w, kept=kept, new=new, err=int(err.item()))


def dst_table(case, budget):
    n = -(-budget // case.page)
    dst = torch.full((len(case.ctx), n), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(case.ctx):
        if c > budget:
            dst[b] = torch.tensor(case.spare[at:at + n], dtype=torch.int32)
            at += n
    return dst


def check_evict(case, w, budget, first, recent):
    dst = dst_table(case, budget)
    got = run_evict(case, w, budget, first, recent, dst)
    assert got["err"] == 0
    names = [n for n in ("k", "ks", "v", "vs") if getattr(case, n) is not None]
    want = {n: getattr(case, n).clone() for n in names}
    ww = w.clone()
    kept = torch.full(got["kept"].shape, -1, dtype=torch.int32)
    for b, c in enumerate(case.ctx):
        for h in range(case.kv_heads):
            t = [float(w[int(case.table[b, p // case.page]), h, p % case.page]) for p in range(c)]
            keep = R.select(t, budget, first, recent)
            if keep is None:
                continue
            kept[b, h] = torch.tensor(keep, dtype=torch.int32)
            for i, p in enumerate(keep):
                sp, ss = int(case.table[b, p // case.page]), p % case.page
                dp, ds = int(dst[b, i // case.page]), i % case.page
                for n in names:
                    src = getattr(case, n)
                    if case.layout == NHD:
                        want[n][dp, ds, h] = src[sp, ss, h]
                    else:
                        want[n][dp, h, ds] = src[sp, h, ss]
                ww[dp, h, ds] = w[sp, h, ss]
    assert torch.equal(got["kept"].cpu(), kept)
    assert got["new"].tolist() == [min(c, budget) for c in case.ctx]
    for n in names:
        assert same(got[n], want[n]), n
    assert same(got["w"], ww)


@pytest.mark.parametrize("kv", [BF16, MX4])
@pytest.mark.parametrize("layout,dim,kv_heads,page,ctx,budget,first,recent", [
    (NHD, 128, 2, 16, [100, 40, 20, 0], 33, 1, 5),
    (HND, 64, 3, 32, [257, 64, 65], 64, 4, 16),
    (NHD, 64, 1, 16, [2, 1], 1, 0, 0),
    (HND, 128, 1, 64, [500], 130, 0, 130),
    (NHD, 64, 2, 128, [300, 131], 130, 130, 0),
    (NHD, 64, 1, 16, [3000], 1500, 3, 100),
])
def test_evict_against_the_plain_form(kv, layout, dim, kv_heads, page, ctx, budget, first, recent):
    spare = sum(c > budget for c in ctx) * -(-budget // page)
    case = R.Case(ctx, [0] * len(ctx), heads=kv_heads, kv_heads=kv_heads, dim=dim, page=page,
                  layout=layout, kv=kv, seed=31, spare=spare)
    g = torch.Generator().manual_seed(2)
    w = torch.floor(torch.rand((case.num_pages, kv_heads, page), generator=g) * 50) / 7
    check_evict(case, w, budget, first, recent)


def test_evict_orders_every_kind_of_weight():
    """Equal weights everywhere, both zeros, infinities, negatives, subnormals, NaN."""
    n, budget = 90, 40
    case = R.Case([n], [0], heads=1, kv_heads=1, dim=64, page=16, kv=BF16, seed=32, spare=3)
    case.k, case.v = torch.nan_to_num(case.k), torch.nan_to_num(case.v)
    w = torch.full((case.num_pages, 1, 16), 0.5)
    check_evict(case, w, budget, 0, 0)
    vals = [math.nan, math.inf, -math.inf, 0.0, -0.0, 1e-42, -1e-42, 1.0, -1.0, 3.0e38]
    for i in range(n):
        w[int(case.table[0, i // 16]), 0, i % 16] = vals[i % len(vals)]
    for budget in (5, 20, 40, 47, 81):
        c = R.Case([n], [0], heads=1, kv_heads=1, dim=64, page=16, kv=BF16, seed=32, spare=6)
        w = torch.zeros((c.num_pages, 1, 16))
        for i in range(n):
            w[int(c.table[0, i // 16]), 0, i % 16] = vals[i % len(vals)]
        check_evict(c, w, budget, 2, 3)


def test_evict_longer_than_shared_memory_holds():
    n, budget = 60000, 777
    case = R.Case([5, n], [0, 0], heads=1, kv_heads=1, dim=64, page=256, kv=MX4, seed=33, spare=4)
    g = torch.Generator().manual_seed(3)
    w = torch.floor(torch.rand((case.num_pages, 1, 256), generator=g) * 3000)
    dst = dst_table(case, budget)
    got = run_evict(case, w, budget, 4, 32, dst)
    assert got["err"] == 0
    t = [float(w[int(case.table[1, p // 256]), 0, p % 256]) for p in range(n)]
    keep = R.select(t, budget, 4, 32)
    assert got["kept"][1, 0].tolist() == keep
    rows = case.get(case.k, 1, n)[torch.tensor(keep)]
    assert same(case.get(got["k"].cpu(), 1, budget, dst), rows)


@pytest.mark.parametrize("n,kinds", [
    (5000, 1),          # all equal: more of the threshold's upper half than are listed
    (5000, 3), (5000, 1 << 20),
    (3000, 2),          # the same for short sequences
    (100003, 5), (100003, 1 << 20),     # upper halves do not fit shared memory
])
def test_evict_of_many_equal_and_of_very_many_keys(n, kinds):
    budget, first, recent, page = 1537, 5, 21, 256
    g = torch.Generator().manual_seed(n + kinds)
    pages = -(-n // page) + -(-budget // page)
    perm = torch.randperm(pages, generator=g).int()
    need = -(-n // page)
    table, dst = perm[:need].view(1, -1).cuda(), perm[need:].view(1, -1).cuda()
    # (halves of the mantissa differ, so that upper halves of the keys repeat)
    w = torch.randint(0, kinds, (pages, 1, page), generator=g).float() * 1e-3 + 2.0
    k = torch.arange(pages * page * 32, dtype=torch.int32).view(torch.int16).view(torch.bfloat16)
    k = k.view(pages, page, 1, 64).cuda()
    v = k.flip(0).contiguous()
    p = B.PaProblem(num_seqs=1, num_q_heads=1, num_kv_heads=1, head_dim=64, page_size=page,
                    num_pages=pages, max_pages_per_seq=need, max_context_len=n, kv_dtype=BF16,
                    sm_scale=1.0)
    ctx = torch.tensor([n], dtype=torch.int32, device="cuda")
    new = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept = torch.zeros((1, 1, budget), dtype=torch.int32, device="cuda")
    err, wd = error_word(), w.cuda()
    old_k = k.view(torch.int16)[table[0].long()].reshape(-1, 64)
    old_v = v.view(torch.int16)[table[0].long()].reshape(-1, 64)
    B.pa_kv_evict(p, budget, first, recent, k, None, v, None, wd, table, dst, ctx, kept, new, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and int(new.item()) == budget
    line = w[table[0].cpu().long()].reshape(-1)[:n].clone()
    line[:first] = math.inf
    line[n - recent:] = math.inf
    want = torch.sort(torch.sort(-line, stable=True).indices[:budget]).values
    assert torch.equal(kept.cpu().view(-1).long(), want)
    for cache, old in ((k, old_k), (v, old_v)):
        got = cache.view(torch.int16)[dst[0].long()].reshape(-1, 64)[:budget]
        assert torch.equal(got, old[want.cuda()])
    got = wd[dst[0].long()].reshape(-1)[:budget].cpu()
    assert torch.equal(got, w[table[0].cpu().long()].reshape(-1)[want])


def test_evict_flags_bad_input():
    case = R.Case([100, 60], [0, 0], heads=1, kv_heads=1, dim=64, page=16, kv=BF16, seed=34, spare=4)
    w = torch.rand((case.num_pages, 1, 16))
    dst = dst_table(case, 20)
    clean = run_evict(case, w, 20, 0, 0, dst)
    bad = dst.clone()
    bad[0, 1] = case.num_pages
    got = run_evict(case, w, 20, 0, 0, bad)
    assert got["err"] == B.PA_DEV_BAD_PAGE
    assert same(case.get(got["k"].cpu(), 1, 20, dst), case.get(clean["k"].cpu(), 1, 20, dst))
    assert same(case.get(got["k"].cpu(), 0, 16, dst), case.get(clean["k"].cpu(), 0, 16, dst))
    case.ctx[0] = 1000                                 # above the declared maximum
    got = run_evict(case, w, 20, 0, 0, dst, max_context_len=100)
    assert got["err"] == B.PA_DEV_BAD_LENGTHS and got["new"].tolist() == [0, 20]


# ----------------------------------------------------------------- together

@pytest.mark.parametrize("kv", [BF16, MX4])
def test_a_serving_run(kv):
    """Prompts written, observed, evicted to a budget; then decode steps over
    what is left: every step's attention equals the plain form over the rows
    that the caches hold."""
    budget, page, heads, kv_heads, dim = 40, 16, 4, 2, 64
    case = R.Case([120, 35], [120, 35], heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                  layout=HND, kv=kv, seed=41, spare=8)
    (k, ks), (v, vs) = case.empty(), case.empty()
    k, ks, v, vs = dev(k), dev(ks), dev(v), dev(vs)
    w = torch.full((case.num_pages, kv_heads, page), 3.0, device="cuda")
    c, q = case.lens()
    err = error_word()
    table = dev(case.table)
    B.pa_kv_append(case.problem(B), new_rows(case, case.kd).cuda(), new_rows(case, case.vd).cuda(),
                   table, c, q, k, ks, v, vs, w, err)
    # the last 8 queries of each prompt observe it
    case.ql = [8, 8]
    case.total_q = 16
    case.q = case.q[-16:]
    lse = R.attention(case)[1].float()
    _, q8 = case.lens()
    B.pa_key_weights(case.problem(B), case.q.cuda(), k, ks, table, c, q8, lse.cuda(), w, err)
    n = 4                                       # pages: the budget and the steps after it
    dst = torch.full((2, max(n, case.mpps)), -1, dtype=torch.int32)
    dst[0, :n] = torch.tensor(case.spare[:n], dtype=torch.int32)
    kept = torch.full((2, kv_heads, budget), -1, dtype=torch.int32, device="cuda")
    new = torch.zeros(2, dtype=torch.int32, device="cuda")
    B.pa_kv_evict(case.problem(B), budget, 2, 8, k, ks, v, vs, w, table, dev(dst), c, kept, new,
                  err)
    torch.cuda.synchronize()
    assert new.tolist() == [40, 35] and int(err.item()) == 0
    add, _ = R.key_weights(case, lse)
    for h in range(kv_heads):
        got = set(kept[0, h].tolist())
        assert len(got) == budget and {0, 1} <= got and set(range(112, 120)) <= got
        # every evicted key has no more weight than every kept, unprotected one
        out = [float(add[0][h, p]) for p in range(2, 112) if p not in got]
        keep = [float(add[0][h, p]) for p in range(2, 112) if p in got]
        assert max(out) <= min(keep) * (1 + 1e-4)
    table2 = case.table.clone()
    table2[0] = dst[0, :case.mpps]
    case.table = table2
    ctx = [40, 35]
    for step in range(3):
        ctx = [x + 1 for x in ctx]
        rows = torch.randn((2, kv_heads, dim), generator=torch.Generator().manual_seed(step))
        rows = rows.to(torch.bfloat16).cuda()
        s = R.Case(ctx, [1, 1], heads=heads, kv_heads=kv_heads, dim=dim, page=page, layout=HND,
                   kv=kv, seed=50 + step)
        s.table, s.mpps, s.num_pages = case.table, case.mpps, case.num_pages
        p = s.problem(B)
        cl, qlen = s.lens()
        B.pa_kv_append(p, rows, rows, dev(s.table), cl, qlen, k, ks, v, vs, w, err)
        if kv == MX4:
            ws = torch.zeros(B.pa_mx4_workspace_size(p), dtype=torch.uint8, device="cuda")
            out = torch.empty((2, heads, dim), dtype=torch.bfloat16, device="cuda")
            lse = torch.empty((2, heads), device="cuda")
            B.pa_decode_mx4(p, s.q.cuda(), k, ks, v, vs, dev(s.table), cl, qlen, ws, out, lse)
        else:
            bufs = B.Buffers(p, B.PA_MODE_DECODE, "cuda", 2, heads, dim)
            B.pa_assign(p, B.PA_MODE_DECODE, cl, qlen, None, bufs.assign_ws)
            B.pa_decode_splitk(p, s.q.cuda(), k, v, dev(s.table), cl, qlen, None, None,
                               bufs.assign_ws, bufs.partial_ws, bufs.out, bufs.lse)
            out, lse = bufs.out, bufs.lse
        B.pa_key_weights(p, s.q.cuda(), k, ks, dev(s.table), cl, qlen, lse, w, err)
        torch.cuda.synchronize()
        s.k, s.v = k.cpu(), v.cpu()
        s.ks, s.vs = (None, None) if ks is None else (ks.cpu(), vs.cpu())
        ref, rl, mag, big = R.attention(s)
        # bf16 probabilities (2^-8) in the bf16 decode, f16 in the 4-bit one
        tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 if kv == BF16 else 2.0 ** -10) * mag + 1e-6
        assert bool(((out.cpu().double() - ref).abs() <= tol).all())
        assert float((lse.cpu().double() - rl).abs().max()) < 1e-4
    assert int(err.item()) == 0


def test_expanded_pages_feed_prefill():
    """A prompt's first part kept in 4 bits, read back as bf16 pages, and its
    second part's prefill over them."""
    case = R.Case([300, 90], [100, 90], heads=4, kv_heads=2, dim=64, page=32, seed=42)
    p = case.problem(B)
    p.kv_dtype = BF16
    c, q = case.lens()
    full = case.problem(B, total_q_tokens=390, max_q_len=300)
    k, v = (torch.zeros(case.shape(64), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    err = error_word()
    t = dev(case.table)
    B.pa_kv_expand(full, dev(case.k), dev(case.ks), dev(case.v), dev(case.vs), t, c, c, t,
                   case.num_pages, k, v, err)
    bufs = B.Buffers(p, B.PA_MODE_PREFILL, "cuda", case.total_q, 4, 64)
    B.pa_assign(p, B.PA_MODE_PREFILL, c, q, None, bufs.assign_ws)
    B.pa_prefill(p, case.q.cuda(), k, v, t, c, q, None, None, None, bufs.assign_ws,
                 bufs.partial_ws, bufs.out, bufs.lse)
    B.pa_combine(p, B.PA_MODE_PREFILL, bufs.assign_ws, bufs.partial_ws, bufs.out, bufs.lse)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    ref, rl, mag, _ = R.attention(case)
    tol = 2.0 ** -8 * ref.abs() + 2.0 ** -8 * mag + 1e-6
    assert bool(((bufs.out.cpu().double() - ref).abs() <= tol).all())


def test_a_captured_step_replays_on_new_lengths():
    """Append, decode and weights captured once; replayed after the lengths in
    device memory moved on."""
    case = R.Case([50, 17], [1, 1], heads=4, kv_heads=2, dim=128, page=16, seed=43)
    case.table = torch.arange(10, dtype=torch.int32).reshape(2, 5)
    case.mpps, case.num_pages = 5, 10
    case.fill()
    p = case.problem(B, max_context_len=80)
    k, ks, v, vs = dev(case.k), dev(case.ks), dev(case.v), dev(case.vs)
    c, q = case.lens()
    t, qs = dev(case.table), case.q.cuda()
    rows = torch.randn((2, 2, 128)).to(torch.bfloat16).cuda()
    ws = torch.zeros(B.pa_mx4_workspace_size(p), dtype=torch.uint8, device="cuda")
    out = torch.zeros((2, 4, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((2, 4), device="cuda")
    w = torch.zeros((10, 2, 16), device="cuda")
    err = error_word()

    def step():
        B.pa_kv_append(p, rows, rows, t, c, q, k, ks, v, vs, None, err)
        B.pa_decode_mx4(p, qs, k, ks, v, vs, t, c, q, ws, out, lse)
        B.pa_key_weights(p, qs, k, ks, t, c, q, lse, w, err)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        c += 1
        rows.copy_(torch.randn((2, 2, 128)).to(torch.bfloat16))
        w.zero_()
        graph.replay()
        torch.cuda.synchronize()
        case.ctx = c.tolist()
        case.k, case.ks, case.v, case.vs = k.cpu(), ks.cpu(), v.cpu(), vs.cpu()
        ref, rl, mag, big = R.attention(case)
        tol = 2.0 ** -8 * ref.abs() + 2.0 ** -10 * mag + 1e-6
        assert bool(((out.cpu().double() - ref).abs() <= tol).all())
        # a softmax row's weights sum to one per q head
        assert abs(float(w.sum()) - 8.0) < 1e-4
    assert int(err.item()) == 0


def test_a_captured_observation_and_eviction_replay_on_new_lengths():
    """Weights of many query rows and the eviction that follows, captured once
    (two kernels of which overlap), replayed with other lengths and queries:
    bit for bit what eager calls give."""
    page, budget, hk = 16, 70, 2
    case = R.Case([400, 290, 130], [12, 12, 12], heads=8, kv_heads=hk, dim=64, page=page, kv=MX4,
                  seed=61, spare=15)
    p = case.problem(B)
    dst = torch.tensor(case.spare, dtype=torch.int32).view(3, 5).cuda()
    k, ks, v, vs = dev(case.k), dev(case.ks), dev(case.v), dev(case.vs)
    base = [x.clone() for x in (k, ks, v, vs)]
    c, q = case.lens()
    t, qs = dev(case.table), case.q.cuda()
    lse = torch.full((36, 8), 4.0, device="cuda")
    w = torch.zeros((case.num_pages, hk, page), device="cuda")
    kept = torch.zeros((3, hk, budget), dtype=torch.int32, device="cuda")
    new = torch.zeros(3, dtype=torch.int32, device="cuda")
    err = error_word()

    def reset():
        for x, y in zip((k, ks, v, vs), base):
            x.copy_(y)
        w.zero_()
        kept.zero_()

    def step():
        B.pa_key_weights(p, qs, k, ks, t, c, q, lse, w, err)
        B.pa_kv_evict(p, budget, 4, 8, k, ks, v, vs, w, t, dst, c, kept, new, err)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([400, 290, 130], [333, 64, 71], [70, 250, 12]):
        c.copy_(torch.tensor(lens, dtype=torch.int32))
        qs.copy_(torch.randn(tuple(qs.shape)).to(torch.bfloat16))
        got = []
        for run in (graph.replay, step):
            reset()
            run()
            torch.cuda.synchronize()
            got.append([x.clone() for x in (w, kept, new, k, ks, v, vs)])
        assert new.tolist() == [min(x, budget) for x in lens]
        for a, b in zip(*got):
            assert same(a, b)
    assert int(err.item()) == 0
