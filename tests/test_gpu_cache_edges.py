"""The cache operators (include/pa_cache.h) where they can go wrong quietly:
workspaces shared by calls of different grids, the smallest scales, a key that
outweighs all others, pages that are none, and the variants that only many or
long sequences reach.  References in 64 bits; the tolerances are those of
test_gpu_cache.py, with what a case adds to them derived beside it.
"""
import math

import pytest
import torch

from paged_attention_gb300 import binding as B

import cache_ref as R
from test_gpu_cache import (BF16, HND, MX4, NHD, check_decode, check_weights, decode, dst_table,
                            error_word, run_evict, run_weights, same)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------- caches of random codes

class Coded:
    """A 4-bit cache of random codes and scales on the device; sequence b holds
    lens[b] tokens in pages of its own."""

    def __init__(self, lens, ql, *, heads, kv_heads, dim, page=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.ql = lens, ql
        self.heads, self.kv_heads, self.dim, self.page = heads, kv_heads, dim, page
        need = [-(-n // page) for n in lens]
        self.pages, self.mpps = sum(need), max(need)
        perm = torch.randperm(self.pages, generator=g, device="cuda").int()
        self.table = torch.full((len(lens), self.mpps), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        shape = (self.pages, page, kv_heads)

        def bytes_(last, lo, hi):
            return torch.randint(lo, hi, shape + (last,), generator=g, device="cuda",
                                 dtype=torch.uint8)

        self.k, self.v = bytes_(dim // 2, 0, 256), bytes_(dim // 2, 0, 256)
        self.ks, self.vs = bytes_(dim // 32, 123, 127), bytes_(dim // 32, 122, 128)
        self.q = torch.randn((sum(ql), heads, dim), generator=g, device="cuda").to(torch.bfloat16)
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.ctx_t, self.ql_t = ints(lens), ints(ql)

    def problem(self, **kw):
        p = B.PaProblem(num_seqs=len(self.lens), num_q_heads=self.heads,
                        num_kv_heads=self.kv_heads, head_dim=self.dim, page_size=self.page,
                        num_pages=self.pages, max_pages_per_seq=self.mpps,
                        total_q_tokens=sum(self.ql), max_q_len=max(self.ql),
                        max_context_len=max(self.lens), kv_dtype=MX4, sm_scale=self.dim ** -0.5)
        for k, v in kw.items():
            setattr(p, k, v)
        return p

    def decode(self, ws, **kw):
        out = torch.full((sum(self.ql), self.heads, self.dim), 7.0, dtype=torch.bfloat16,
                         device="cuda")
        lse = torch.full(out.shape[:2], 7.0, device="cuda")
        B.pa_decode_mx4(self.problem(**kw), self.q, self.k, self.ks, self.v, self.vs, self.table,
                        self.ctx_t, self.ql_t, ws, out, lse)
        return out, lse

    def space(self, **kw):
        return torch.zeros(B.pa_mx4_workspace_size(self.problem(**kw)), dtype=torch.uint8,
                           device="cuda")

    def rows(self, which, b):
        cache, sc = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        pages = self.table[b][:-(-self.lens[b] // self.page)].long()
        x, s = (t[pages].reshape(-1, self.kv_heads, t.shape[-1])[:self.lens[b]].cpu()
                for t in (cache, sc))
        return R.dequantise(x, s).cuda()

    def check(self, out, lse):
        """Against 64 bits, with test_gpu_cache.check_decode's tolerances."""
        at, G = 0, self.heads // self.kv_heads
        for b, (n, ql) in enumerate(zip(self.lens, self.ql)):
            K, V = (self.rows(w, b).transpose(0, 1).repeat_interleave(G, 0) for w in "kv")
            q = self.q[at:at + ql].double().transpose(0, 1)
            hide = (torch.arange(n, device="cuda")[None]
                    > torch.arange(n - ql, n, device="cuda")[:, None])
            x = (q @ K.transpose(1, 2) * self.dim ** -0.5).masked_fill(hide, -math.inf)
            big = (q.abs() @ K.abs().transpose(1, 2)).amax(-1) * self.dim ** -0.5
            p = torch.softmax(x, -1)
            ref, mag, rl = p @ V, p @ V.abs(), torch.logsumexp(x, -1)
            score = (self.dim + 8) * 2.0 ** -24 * big
            tol = 2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2.0 ** -14 + 2 * score[..., None]) * mag
            d = (out[at:at + ql].double().transpose(0, 1) - ref).abs()
            assert bool((d <= tol + 1e-30).all()), float((d / tol).max())
            dl = (lse[at:at + ql].double().t() - rl).abs()
            assert bool((dl <= score + 2.0 ** -20 + rl.abs() * 2.0 ** -21).all())
            at += ql


# ---------------------------------------------------------------- workspaces

@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("grid", [1, 8, 152])
def test_one_workspace_serves_grids_of_any_size(dim, grid):
    """A call of few CTAs, then one of the most there can be, in turn in one
    workspace: every call gives what a fresh workspace gives."""
    few = Coded([3000, 900], [1, 1], heads=8, kv_heads=1, dim=dim, seed=1)
    # units that begin in every part of the grid and are split
    many = Coded([40000], [1], heads=8, kv_heads=8, dim=64, seed=2)
    a, b = dict(num_ctas=grid, unit_cost=-1), dict(num_ctas=1024, unit_cost=-1)
    want_few, want_many = few.decode(few.space(**a), **a), many.decode(many.space(**b), **b)
    ws = torch.zeros(max(few.space(**a).numel(), many.space(**b).numel()), dtype=torch.uint8,
                     device="cuda")
    for _ in range(3):
        got = few.decode(ws, **a)
        assert torch.equal(got[0], want_few[0]) and torch.equal(got[1], want_few[1])
        got = many.decode(ws, **b)
        assert torch.equal(got[0], want_many[0]) and torch.equal(got[1], want_many[1])
    assert B.pa_last_device_error(ws) == 0


@pytest.mark.parametrize("fill", [0x7F, 0xFF])
def test_a_workspace_that_does_not_start_as_zeros_is_reported(fill):
    """Counters that no call leaves behind: reported, where rows would go
    missing silently; zeros make the workspace good again."""
    c = Coded([5000], [1], heads=8, kv_heads=1, dim=64, seed=14)
    want = c.decode(c.space())
    ws = c.space()
    ws[256:256 + 4 * 1024] = fill
    c.decode(ws)
    assert B.pa_last_device_error(ws) == B.PA_DEV_BAD_WORKSPACE
    ws.zero_()
    got = c.decode(ws)
    assert B.pa_last_device_error(ws) == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_decode_repeats_itself_bit_for_bit():
    """Calls after calls of a batch whose units are split over CTAs."""
    c = Coded([128, 20000, 333, 4500, 64, 9000], [2, 2, 1, 2, 2, 1], heads=32, kv_heads=8, dim=128,
              seed=3)
    ws = c.space()
    first = c.decode(ws)
    c.check(*first)
    for i in range(10):
        got = c.decode(ws if i % 2 else c.space())
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


@pytest.mark.parametrize("dim,heads,n", [(64, 1, 20011), (128, 3, 70001), (128, 32, 9001)])
def test_decode_of_one_unit_over_many_ctas(dim, heads, n):
    """One KV head: its parts are joined 32 at a time, several times over (32
    heads: as two blocks of rows)."""
    c = Coded([n], [1], heads=heads, kv_heads=1, dim=dim, seed=4)
    c.check(*c.decode(c.space()))
    c.check(*c.decode(c.space(num_ctas=1024, unit_cost=-1), num_ctas=1024, unit_cost=-1))


# --------------------------------------------------------------------- scales

@pytest.mark.parametrize("dim", [64, 128])
def test_the_smallest_scale_counts(dim):
    """Blocks of K with scale byte 0 are codes times 2^-127, as the format says,
    for queries near the top of bf16's range.  (bf16 queries are exact in f16
    with their power of two taken out; a score's rounding in the subnormal range
    is 2^-150, times a factor below 2^120: nothing beside the tolerance.)"""
    case = R.Case([70, 33], [2, 1], heads=4, kv_heads=2, dim=dim, seed=5)
    g = torch.Generator().manual_seed(5)
    q = torch.randn(case.q.shape, generator=g).clamp(-3.5, 3.5)
    case.q = (q * 2.0 ** 125).to(torch.bfloat16)
    poison = case.ks == 255
    case.ks = torch.randint(0, 3, case.ks.shape, generator=g, dtype=torch.uint8)
    case.ks[poison] = 255
    check_decode(case)
    # whole rows of scale 0
    case.ks = torch.where(poison, 255, 0).to(torch.uint8)
    out, lse = check_decode(case)
    assert float(lse.std()) > 1e-3                 # scores that are not all 0
    # the key weights of the same cache agree with that lse
    _, rl, _, _ = R.attention(case)
    w, err = run_weights(case, lse.cpu().double(), torch.zeros((case.num_pages, 2, 16)))
    assert err == 0 and abs(float(w.sum()) - 3 * 4) < 1e-4


# ------------------------------------------------------------------- softmax

@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("above", [9.0, 12.0, 18.0])
@pytest.mark.parametrize("where", [0, 40])
def test_a_key_that_outweighs_the_others_and_has_no_value(dim, above, where):
    """What is left of the output is the others' values.  A probability rounds
    to f16 after a factor 2^7 and relative to a maximum that is at most the
    row's: below f16's normal range it is off by at most 2^-25 / 2^7 = 2^-32 of
    the largest probability, so the output by 2^-32 of the sum of |v|."""
    g = torch.Generator().manual_seed(6)
    case = R.Case([300], [1], heads=1, kv_heads=1, dim=dim, seed=6, kmag=0.02)
    q = case.q[0, 0].float()
    case.kd[0][where, 0] = (q * (above * math.sqrt(dim) / float(q @ q))).to(torch.bfloat16)
    case.vd[0][where] = 0
    case.fill()
    out, lse, ws = decode(case)
    assert B.pa_last_device_error(ws) == 0
    ref, rl, mag, big = R.attention(case)
    assert float((R.key_weights(case, rl)[0][0][0, where])) > 0.9
    score = (dim + 8) * 2.0 ** -24 * big
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2.0 ** -14 + 2 * score[..., None]) * mag
    tol = tol + 2.0 ** -32 * case.rows("v", 0)[:, 0].abs().sum(0)
    d = (out.cpu().double() - ref).abs()
    assert bool((d <= tol).all()), f"out off by {float((d / tol).max())} of its tolerance"
    d = (lse.cpu().double() - rl).abs()
    assert bool((d <= score + 2.0 ** -20 + rl.abs() * 2.0 ** -21).all())


# ------------------------------------------------------------------ bad pages

def attention_without(case, hidden):
    """R.attention (out, lse, sum p |v|, largest sum |q k|) where sequence b's
    keys at positions hidden[b] are not there."""
    T, H, D, G = case.total_q, case.heads, case.dim, case.group
    out, mag = torch.zeros((2, T, H, D), dtype=torch.float64)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64)
    big = torch.zeros((T, H), dtype=torch.float64)
    at = 0
    for b, (c, q) in enumerate(zip(case.ctx, case.ql)):
        K, V = case.rows("k", b), case.rows("v", b)
        for i in range(q):
            p = c - q + i
            lo = max(0, p - case.window + 1) if case.window else 0
            see = [j for j in range(lo, p + 1) if j not in hidden[b]]
            for h in range(H):
                if not see:
                    continue
                k, v, x = K[see, h // G], V[see, h // G], case.q[at + i, h].double()
                s = (k @ x) * case.scale
                lse[at + i, h] = torch.logsumexp(s, 0)
                out[at + i, h] = torch.softmax(s, 0) @ v
                mag[at + i, h] = torch.softmax(s, 0) @ v.abs()
                big[at + i, h] = (k.abs() @ x.abs()).max() * case.scale
        at += q
    return out, lse, mag, big


@pytest.mark.parametrize("dim,heads,kv_heads,page,layout,window,bad", [
    (64, 2, 1, 16, NHD, 0, [(0, 2), (0, 5)]),             # first and second halves of a step
    (128, 8, 2, 16, HND, 0, [(0, 6), (1, 0), (1, 2), (1, 1)]),
    (128, 4, 1, 64, NHD, 0, [(0, 1), (1, 0)]),            # sequence 1: every key
    (64, 4, 4, 32, HND, 40, [(0, 3), (1, 1)]),            # some queries see no other page
    (128, 16, 1, 16, NHD, 0, [(0, 0), (0, 6)]),           # two blocks of rows
])
@pytest.mark.parametrize("entry", [-1, 1 << 30])
def test_decode_leaves_out_the_keys_of_a_bad_page(dim, heads, kv_heads, page, layout, window, bad,
                                                  entry):
    """Keys whose page is outside the pool are not there; a query that sees no
    other gets zeros and lse -inf; the error word tells."""
    case = R.Case([100, 50], [2, 2], heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                  layout=layout, window=window, seed=7)
    hidden = [set(), set()]
    for b, i in bad:
        hidden[b].update(range(i * page, (i + 1) * page))
    ref, rl, mag, big = attention_without(case, hidden)
    for b, i in bad:
        case.table[b, i] = entry
    score = (dim + 8) * 2.0 ** -24 * big
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2.0 ** -14 + 2 * score[..., None]) * mag
    for kw in (dict(), dict(num_ctas=1), dict(num_ctas=1024, unit_cost=-1)):
        out, lse, ws = decode(case, **kw)
        assert B.pa_last_device_error(ws) == B.PA_DEV_BAD_PAGE
        assert bool(((out.cpu().double() - ref).abs() <= tol).all())
        none = rl == -math.inf
        assert torch.equal(lse.cpu() == -math.inf, none)
        d = (lse.cpu().double() - rl).abs()[~none]
        assert bool((d <= (score + 2.0 ** -20 + rl.abs() * 2.0 ** -21)[~none]).all())


@pytest.mark.parametrize("kv", [BF16, MX4])
@pytest.mark.parametrize("n,page,where", [(100, 16, 3), (700, 64, 0), (5000, 256, 19)])
def test_evict_flags_a_bad_page_whose_keys_go(kv, n, page, where):
    """The keys of a page that is none are the first to go, and nothing of them
    is moved: the error word tells all the same, and the others are chosen and
    moved as if those had no weight."""
    budget = n // 3
    case = R.Case([n, 20], [0, 0], heads=2, kv_heads=2, dim=64, page=page, kv=kv, seed=8,
                  spare=-(-budget // page))
    w = torch.rand((case.num_pages, 2, page), generator=torch.Generator().manual_seed(8)) + 0.1
    dst = dst_table(case, budget)
    no_weight = w.clone()
    no_weight[int(case.table[0, where])] = math.nan
    clean = run_evict(case, no_weight, budget, 0, 0, dst)
    assert clean["err"] == 0
    for entry in (case.num_pages, -5):
        case.table[0, where] = entry
        got = run_evict(case, w, budget, 0, 0, dst)
        assert got["err"] == B.PA_DEV_BAD_PAGE
        assert torch.equal(got["kept"], clean["kept"]) and torch.equal(got["new"], clean["new"])
        for name in ("k", "ks", "v", "vs"):
            if clean[name] is not None:
                assert same(got[name], clean[name]), name
        assert same(got["w"][dst[0].long()], clean["w"][dst[0].long()])


# ------------------------------------------------- eviction of many and of long

def plain_kept(line, n, budget, first, recent):
    """Positions kept of weights line[..., n], ascending."""
    x = line.clone()
    x[..., :first] = math.inf
    x[..., n - recent:] = math.inf
    return torch.sort(torch.sort(-x, dim=-1, stable=True).indices[..., :budget]).values


@pytest.mark.parametrize("batch,kv_heads,most,budget,page,kinds,kv", [
    (40, 4, 1100, 700, 64, 1 << 20, BF16),
    (40, 4, 6000, 1000, 64, 1 << 20, BF16),       # more pairs than SMs, up to 12288 keys
    (40, 4, 6000, 1000, 64, 3, MX4),
    (40, 4, 13000, 2000, 64, 1 << 20, MX4),       # and above
    (40, 4, 13000, 2000, 64, 3, BF16),
    (3, 3, 100003, 3001, 256, 1 << 20, MX4),      # upper halves that do not fit shared memory
    (60, 3, 97001, 130, 128, 5, BF16),            # the same, more pairs than SMs
    (60, 3, 94000, 130, 128, 1 << 20, MX4),       # just past what fits
])
def test_evict_of_many_and_of_long_sequences(batch, kv_heads, most, budget, page, kinds, kv):
    g = torch.Generator(device="cuda").manual_seed(most)
    first, recent, dim = 4, 40, 64
    lens = torch.randint(most // 2, most + 1, (batch,), generator=g, device="cuda")
    lens[0] = most
    lens[1] = budget                              # one that stays
    need, keep = -(-most // page), -(-budget // page)
    pages = batch * (need + keep)
    perm = torch.randperm(pages, generator=g, device="cuda").int().view(batch, need + keep)
    table, dst = perm[:, :need].contiguous(), perm[:, need:].contiguous()
    # (halves of the mantissa differ, so that upper halves of the keys repeat)
    w = torch.randint(0, kinds, (pages, kv_heads, page), generator=g, device="cuda") * 1e-3 + 2
    row = dim if kv == BF16 else dim // 2
    t = torch.int16 if kv == BF16 else torch.uint8

    def cache(last):
        return torch.randint(0, 100, (pages, page, kv_heads, last), generator=g, device="cuda",
                             dtype=torch.int32).to(t)

    k, v = cache(row), cache(row)
    ks, vs = (cache(2), cache(2)) if kv == MX4 else (None, None)
    p = B.PaProblem(num_seqs=batch, num_q_heads=kv_heads, num_kv_heads=kv_heads, head_dim=dim,
                    page_size=page, num_pages=pages, max_pages_per_seq=need, max_context_len=most,
                    kv_dtype=kv, sm_scale=1.0)
    ctx = lens.int()
    new = torch.full((batch,), -1, dtype=torch.int32, device="cuda")
    kept = torch.full((batch, kv_heads, budget), -1, dtype=torch.int32, device="cuda")
    err, old = error_word(), [x.clone() for x in (k, ks, v, vs) if x is not None] + [w.clone()]
    as_given = (lambda x: x.view(torch.bfloat16)) if kv == BF16 else (lambda x: x)
    B.pa_kv_evict(p, budget, first, recent, as_given(k), ks, as_given(v), vs, w, table, dst, ctx,
                  kept, new, err)
    torch.cuda.synchronize()
    assert int(err) == 0 and torch.equal(new, ctx.clamp(max=budget))
    assert bool((kept[1] == -1).all())
    heads = torch.arange(kv_heads, device="cuda")[:, None]
    at = torch.arange(budget, device="cuda")
    now = [x for x in (k, ks, v, vs) if x is not None]
    for b in range(batch):
        n = int(lens[b])
        if n <= budget:
            continue
        line = old[-1][table[b].long()].transpose(0, 1).reshape(kv_heads, -1)[:, :n]
        want = plain_kept(line, n, budget, first, recent)
        assert torch.equal(kept[b].long(), want)
        sp, dp = table[b].long()[want // page], dst[b].long()[at // page].expand_as(want)
        for got, was in zip(now, old):
            assert torch.equal(got[dp, at % page, heads], was[sp, want % page, heads])
        assert torch.equal(w[dp, heads, at % page], old[-1][sp, heads, want % page])


# ---------------------------------------------------------------- key weights

@pytest.mark.parametrize("kv", [BF16, MX4])
@pytest.mark.parametrize("layout,dim,heads,kv_heads,page,ctx,ql,window", [
    (NHD, 128, 16, 1, 16, [300, 41], [1, 1], 0),              # 16 rows
    (HND, 64, 10, 2, 32, [70, 600, 3], [3, 1, 2], 0),         # 15, 5 and 10 rows
    (NHD, 64, 9, 1, 16, [257, 256], [1, 0], 100),             # 9 rows, a window
    (HND, 128, 4, 2, 64, [90, 513], [8, 5], 33),              # 16 and 10 rows, a window
])
def test_weights_of_two_products_of_rows(kv, layout, dim, heads, kv_heads, page, ctx, ql, window):
    check_weights(R.Case(ctx, ql, heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                         layout=layout, kv=kv, window=window, seed=9))


@pytest.mark.parametrize("kv", [BF16, MX4])
@pytest.mark.parametrize("dim,heads", [(128, 4), (64, 8)])
def test_weights_of_more_items_than_ctas(kv, dim, heads):
    """Few query rows, many sequences and heads: a CTA goes on from item to item,
    over heads and sequences, some of them without queries."""
    g = torch.Generator().manual_seed(10)
    ctx = torch.randint(1, 330, (110,), generator=g).tolist()
    case = R.Case(ctx, [min(c, i % 3) for i, c in enumerate(ctx)], heads=heads, kv_heads=4, dim=dim,
                  page=16, kv=kv, seed=10)
    check_weights(case)


# ------------------------------------------------------------- far pages, scale 0

@pytest.mark.parametrize("kv", [BF16, MX4])
def test_pages_past_32_bits_of_bytes(kv):
    """A pool of more than 2^32 bytes a cache: what the operators do in its last
    pages is what they do in a small pool's."""
    page, hk, G, dim, n, budget = 256, 8, 2, 128, 600, 300
    row = dim * 2 if kv == BF16 else dim // 2
    far = 2 ** 32 // (page * hk * row) + 40
    g = torch.Generator(device="cuda").manual_seed(12)
    rows = torch.randn((2, n, hk, dim), generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn((9, hk * G, dim), generator=g, device="cuda").to(torch.bfloat16)
    lse = torch.full((9, hk * G), 7.0, device="cuda")
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    results = []
    for pages in (8, far):
        table, dst = ints([[pages - 1, pages - 5, pages - 2]]), ints([[pages - 6, pages - 3]])
        p = B.PaProblem(num_seqs=1, num_q_heads=hk * G, num_kv_heads=hk, head_dim=dim,
                        page_size=page, num_pages=pages, max_pages_per_seq=3, total_q_tokens=n,
                        max_q_len=n, max_context_len=n, kv_dtype=kv, sm_scale=dim ** -0.5)
        last, t = (dim, torch.bfloat16) if kv == BF16 else (dim // 2, torch.uint8)
        k, v = (torch.empty((pages, page, hk, last), dtype=t, device="cuda") for _ in "kv")
        ks, vs = ((torch.empty((pages, page, hk, dim // 32), dtype=t, device="cuda") for _ in "kv")
                  if kv == MX4 else (None, None))
        w, err = torch.empty((pages, hk, page), device="cuda"), error_word()
        B.pa_kv_append(p, rows[0], rows[1], table, ints([n]), ints([n]), k, ks, v, vs, w, err)
        got = []
        for ql in (1, 9):                      # few and many query rows
            p.total_q_tokens = p.max_q_len = ql
            B.pa_key_weights(p, q[:ql], k, ks, table, ints([n]), ints([ql]), lse[:ql], w, err)
            if kv == MX4:
                ws = torch.zeros(B.pa_mx4_workspace_size(p), dtype=torch.uint8, device="cuda")
                out = torch.empty((ql, hk * G, dim), dtype=torch.bfloat16, device="cuda")
                B.pa_decode_mx4(p, q[:ql], k, ks, v, vs, table, ints([n]), ints([ql]), ws, out,
                                None)
                got.append(out)
        if kv == MX4:
            p.total_q_tokens = p.max_q_len = n
            back = [torch.empty((far, page, hk, dim // 4), dtype=torch.float64, device="cuda")
                    .view(torch.bfloat16) for _ in "kv"]
            to = ints([[far - 2, far - 1, far - 4]])
            B.pa_kv_expand(p, k, ks, v, vs, table, ints([n]), ints([n]), to, far, *back, err)
            got += [x[to[0].long()].reshape(-1, hk, dim)[:n].clone() for x in back]
            del back
        kept = torch.zeros((1, hk, budget), dtype=torch.int32, device="cuda")
        B.pa_kv_evict(p, budget, 4, 8, k, ks, v, vs, w, table, dst, ints([n]), kept, ints([0]), err)
        got.append(kept)
        for x in (k, ks, v, vs):
            if x is not None:
                got += [x[tab[0].long()].reshape(-1, hk, x.shape[-1])[:m].clone()
                        for tab, m in ((table, n), (dst, budget))]
        got += [w[tab[0].long()].transpose(0, 1).reshape(hk, -1)[:, :m].clone()
                for tab, m in ((table, n), (dst, budget))]
        assert int(err) == 0
        results.append(got)
        del k, v, ks, vs, w
    assert len(results[0]) == len(results[1])
    for a, b in zip(*results):
        assert same(a, b)


@pytest.mark.parametrize("ql", [[1, 2], [20, 3]])
def test_a_scale_of_zero_is_an_even_softmax(ql):
    case = R.Case([100, 50], ql, heads=2, kv_heads=1, dim=64, seed=13)
    case.scale = 0.0
    out, lse = check_decode(case)
    seen = torch.tensor([c - q + i + 1.0 for c, q in zip(case.ctx, ql) for i in range(q)])
    assert torch.allclose(lse.cpu()[:, 0], seen.log(), rtol=1e-6)
    check_weights(case)


# ------------------------------------------------------------------- refusals

def test_what_would_be_misread_is_refused_on_the_device_too():
    """A strided q, lengths on the host or in 64 bits, a slice of a wider block
    table: refused, with nothing launched."""
    c = Coded([100, 30], [1, 1], heads=4, kv_heads=2, dim=64, page=16, seed=11)
    ws, p = c.space(), c.problem()
    out = torch.full((2, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    good = dict(q=c.q, table=c.table, ctx=c.ctx_t, ql=c.ql_t)
    wide_q = torch.zeros((2, 8, 64), dtype=torch.bfloat16, device="cuda")[:, :4]
    wide_table = torch.zeros((2, c.mpps + 3), dtype=torch.int32, device="cuda")[:, :c.mpps]
    for name, t in (("q", wide_q), ("table", wide_table), ("table", c.table.cpu()),
                    ("ctx", c.ctx_t.cpu()), ("ctx", c.ctx_t.long()), ("ql", c.ql_t.long())):
        a = dict(good, **{name: t})
        with pytest.raises(ValueError):
            B.pa_decode_mx4(p, a["q"], c.k, c.ks, c.v, c.vs, a["table"], a["ctx"], a["ql"], ws, out,
                            None)
    torch.cuda.synchronize()
    assert bool((out == 7.0).all())
    B.pa_decode_mx4(p, c.q, c.k, c.ks, c.v, c.vs, c.table, c.ctx_t, c.ql_t, ws, out, None)
    assert torch.equal(out, c.decode(c.space())[0])


def test_the_current_stream_with_and_without_torchs_unnamed_call(monkeypatch):
    assert B._raw_stream is not None
    side = torch.cuda.Stream()
    for raw in (B._raw_stream, None):
        monkeypatch.setattr(B, "_raw_stream", raw)
        assert B._stream(None) == torch.cuda.current_stream().cuda_stream
        with torch.cuda.stream(side):
            assert B._stream(None) == side.cuda_stream
