"""Plain 64-bit forms of the cache operators (include/pa_cache.h), on the CPU.

Written from the definitions, one element or one row at a time where that is
clearer than fast; sizes in the tests are small.
"""
import math

import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
NHD, HND = 0, 1
BF16, MX4 = 0, 2


def quantise(x):
    """x [..., D] -> (codes uint8 [..., D/2], scale bytes uint8 [..., D/32])."""
    D = x.shape[-1]
    xb = x.double().reshape(*x.shape[:-1], D // 32, 32)
    fine = torch.isfinite(xb).all(-1)
    xs = torch.where(fine[..., None], xb, torch.zeros_like(xb))
    amax = xs.abs().amax(-1)
    e = torch.floor(torch.log2(torch.where(amax > 0, amax, torch.ones_like(amax)))) - 2
    e = torch.where(amax > 0, e, torch.full_like(e, -127.0)).clamp(min=-127.0)
    y = xs / torch.exp2(e)[..., None]
    dist = (y.abs().clamp(max=6.0)[..., None] - E2M1).abs()
    # nearest value; of two equally near ones the even code
    near = dist == dist.amin(-1, keepdim=True)
    penalty = torch.tensor([0.0, 1.0] * 4, dtype=torch.float64)
    code = torch.where(near, penalty, torch.full_like(dist, 9.0)).argmin(-1)
    code = code + 8 * torch.signbit(y).long()
    code = torch.where(fine[..., None], code, torch.zeros_like(code))
    byte = torch.where(fine, e + 127, torch.full_like(e, 255.0))
    code = code.reshape(*x.shape[:-1], D // 2, 2)
    return (code[..., 0] + 16 * code[..., 1]).to(torch.uint8), byte.to(torch.uint8)


def dequantise(codes, scales):
    lo, hi = (codes & 15).long(), (codes >> 4).long()
    c = torch.stack((lo, hi), -1).reshape(*codes.shape[:-1], -1)
    v = torch.where(c >= 8, -E2M1[c & 7], E2M1[c & 7])
    e = scales.double()
    f = torch.where(e == 255, torch.full_like(e, math.nan), torch.exp2(e - 127))
    return v * f.repeat_interleave(32, -1)


class Case:
    """A paged cache on the CPU with its lengths; rows of unused slots and
    pages are poisoned (NaN rows, or NaN scales over all-ones codes)."""

    def __init__(self, ctx, ql, *, heads=4, kv_heads=2, dim=128, page=16, layout=NHD, kv=MX4,
                 window=0, seed=0, spare=0, kmag=1.0, vmag=None, q=None):
        g = torch.Generator().manual_seed(seed)
        self.ctx, self.ql = list(ctx), list(ql)
        self.heads, self.kv_heads, self.dim, self.page = heads, kv_heads, dim, page
        self.layout, self.kv, self.window = layout, kv, window
        self.group = heads // kv_heads
        self.scale = 1.0 / math.sqrt(dim)
        B = len(ctx)
        need = [-(-c // page) for c in ctx]
        self.num_pages = sum(need) + spare + 2
        perm = torch.randperm(self.num_pages, generator=g).tolist()
        self.mpps = max(1, max(need))
        self.table = torch.full((B, self.mpps), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
            at += n
        self.spare = perm[at:at + spare]
        self.total_q = sum(ql)
        self.q = (torch.randn((self.total_q, heads, dim), generator=g).to(torch.bfloat16)
                  if q is None else q)
        # dense rows [B][ctx, Hkv, D]
        mag = [1.0] * B if vmag is None else vmag
        self.kd = [(torch.randn((c, kv_heads, dim), generator=g) * kmag).to(torch.bfloat16)
                   for c in ctx]
        self.vd = [(torch.randn((c, kv_heads, dim), generator=g) * m).to(torch.bfloat16)
                   for c, m in zip(ctx, mag)]
        self.fill()

    def shape(self, last):
        return ((self.num_pages, self.page, self.kv_heads, last) if self.layout == NHD
                else (self.num_pages, self.kv_heads, self.page, last))

    def empty(self):
        """(cache, scales) with every slot poisoned."""
        if self.kv == BF16:
            return torch.full(self.shape(self.dim), math.nan, dtype=torch.bfloat16), None
        return (torch.full(self.shape(self.dim // 2), 0xFF, dtype=torch.uint8),
                torch.full(self.shape(self.dim // 32), 0xFF, dtype=torch.uint8))

    def put(self, cache, b, pos, rows, table=None):
        t = (self.table if table is None else table)[b]
        for i, p in enumerate(pos):
            pg, s = int(t[p // self.page]), p % self.page
            if self.layout == NHD:
                cache[pg, s] = rows[i]
            else:
                cache[pg, :, s] = rows[i]

    def get(self, cache, b, n, table=None):
        t = (self.table if table is None else table)[b]
        out = []
        for p in range(n):
            pg, s = int(t[p // self.page]), p % self.page
            out.append(cache[pg, s] if self.layout == NHD else cache[pg, :, s])
        return torch.stack(out) if out else cache.new_zeros((0, self.kv_heads, cache.shape[-1]))

    def fill(self):
        (self.k, self.ks), (self.v, self.vs) = self.empty(), self.empty()
        for b, c in enumerate(self.ctx):
            for dense, cache, scales in ((self.kd[b], self.k, self.ks), (self.vd[b], self.v, self.vs)):
                if self.kv == BF16:
                    self.put(cache, b, range(c), dense)
                else:
                    codes, sc = quantise(dense)
                    self.put(cache, b, range(c), codes)
                    self.put(scales, b, range(c), sc)

    def rows(self, which, b, n=None):
        """Cached K or V rows of sequence b in 64 bits [n, Hkv, D]."""
        n = self.ctx[b] if n is None else n
        cache, sc = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        x = self.get(cache, b, n)
        return x.double() if self.kv == BF16 else dequantise(x, self.get(sc, b, n))

    def problem(self, B, **kw):
        p = B.PaProblem(
            num_seqs=len(self.ctx), num_q_heads=self.heads, num_kv_heads=self.kv_heads,
            head_dim=self.dim, page_size=self.page, num_pages=self.num_pages,
            max_pages_per_seq=self.mpps, total_q_tokens=self.total_q,
            max_q_len=max(self.ql) if self.ql else 0, max_context_len=max(self.ctx),
            layout=self.layout, kv_dtype=self.kv, sm_scale=self.scale, window=self.window)
        for k, v in kw.items():
            setattr(p, k, v)
        return p

    def lens(self, device="cuda"):
        return (torch.tensor(self.ctx, dtype=torch.int32, device=device),
                torch.tensor(self.ql, dtype=torch.int32, device=device))


def attention(case, weights=None):
    """Per row (token, head): out, lse, sum p |v|, and the largest sum |q k| scale
    over keys (what the tolerances scale with).  With `weights` (fp64 dense
    lists [Hkv, ctx] per sequence, lse given) nothing else is returned."""
    T, H, D, G = case.total_q, case.heads, case.dim, case.group
    out = torch.zeros((T, H, D), dtype=torch.float64)
    mag = torch.zeros((T, H, D), dtype=torch.float64)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64)
    big = torch.zeros((T, H), dtype=torch.float64)
    at = 0
    for b, (c, q) in enumerate(zip(case.ctx, case.ql)):
        if q:
            K, V = case.rows("k", b), case.rows("v", b)
        for i in range(q):
            p = c - q + i
            lo = max(0, p - case.window + 1) if case.window else 0
            for h in range(H):
                k, v = K[lo:p + 1, h // G], V[lo:p + 1, h // G]
                x = case.q[at + i, h].double()
                s = (k @ x) * case.scale
                lse[at + i, h] = torch.logsumexp(s, 0)
                w = torch.softmax(s, 0)
                out[at + i, h] = w @ v
                mag[at + i, h] = w @ v.abs()
                big[at + i, h] = (k.abs() @ x.abs()).max() * case.scale
        at += q
    return out, lse, mag, big


def key_weights(case, lse):
    """Per sequence [Hkv, ctx]: the weight the queries give each key, for the
    given lse [T, H]; and the tolerance that goes with each."""
    got, tol = [], []
    at = 0
    for b, (c, q) in enumerate(zip(case.ctx, case.ql)):
        w = torch.zeros((case.kv_heads, c), dtype=torch.float64)
        t = torch.zeros_like(w)
        if q:
            K = case.rows("k", b)
        for i in range(q):
            p = c - q + i
            lo = max(0, p - case.window + 1) if case.window else 0
            for h in range(case.heads):
                l = float(lse[at + i, h])
                if l == -math.inf:
                    continue
                k = K[lo:p + 1, h // case.group]
                x = case.q[at + i, h].double()
                e = torch.exp((k @ x) * case.scale - l)
                big = (k.abs() @ x.abs()) * case.scale
                w[h // case.group, lo:p + 1] += e
                # the score's fp32 sum, the fp32 exponent, and the exponential's own error
                rel = (case.dim + 8) * 2.0 ** -24 * big + (abs(l) + big) * 2.0 ** -22 + 2.0 ** -20
                t[h // case.group, lo:p + 1] += e * rel
        at += q
        got.append(w)
        tol.append(t)
    return got, tol


def select(weights, budget, first, recent):
    """Positions kept of one (sequence, head): the first, the recent, then the
    largest weights, ties to the lower position, NaN below every number."""
    n = len(weights)
    if n <= budget:
        return None
    safe = [i for i in range(n) if i < first or i >= n - recent]
    rest = [i for i in range(n) if first <= i < n - recent]
    rest.sort(key=lambda i: (math.isnan(weights[i]), -weights[i] if not math.isnan(weights[i]) else 0.0, i))
    return sorted(safe + rest[:budget - len(safe)])
