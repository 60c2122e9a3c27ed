"""Measured cases of the cache operators: what a serving loop does with a paged
K/V cache besides attending to it in bf16 or E4M3.

Four paths, each the calls a user's program makes:

  write    new K/V rows go into the 4-bit microscaled cache (E2M1 elements in
           blocks of 32 along head_dim, one power-of-two scale per block) and
           are read back as bf16 pages, the form a chunk's prefill takes them in
  decode   attention of a few new tokens per sequence over that cache
  weights  the attention weight that a set of queries gives to every cached
           key, added to the key's running total
  evict    the keys to keep by those totals, and their rows (K, V and totals)
           packed into other pages

Lengths come from the case (``lens``, ``lo``, ``hi``, ``lens_seed``), values
from the seed.
"""
import math
import random

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases

def listed():
    base = dict(heads=32, kv_heads=8, dim=128, page=64, layout="NHD", window=0, strided=False,
                kv="mx4", q_len=1, q_ragged=False, budget=0, first=0, recent=0)

    def case(name, kind, batch, lens, lo, hi, lens_seed, **kw):
        c = dict(base, name=name, kind=kind, batch=batch, lens=lens, lo=lo, hi=hi,
                 lens_seed=lens_seed)
        c.update(kw)
        return c

    return [
        # one decode step's new rows of 64 running sequences: latency
        case("write_step_64", "write", 64, "log", 128, 32768, 1),
        # a batch of prompts from a fused QKV projection, ragged, 16-token pages
        case("write_prompts_16", "write", 16, "uniform", 257, 2048, 2, q_len=2048, q_ragged=True,
             page=16, strided=True, layout="HND"),
        # the smallest call: a few short sequences, head_dim 64
        case("decode_tiny", "decode", 3, "uniform", 37, 100, 3, heads=4, kv_heads=1, dim=64,
             page=16),
        # ordinary serving batch, lengths over two orders of magnitude, one draft token
        case("decode_64", "decode", 64, "log", 128, 32768, 4, q_len=2),
        # the largest batch: long contexts, 64 heads, two draft tokens
        case("decode_128", "decode", 128, "uniform", 1024, 16384, 5, heads=64, q_len=3,
             layout="HND"),
        # one very long sequence: the cache's length split over the whole GPU
        case("decode_long_1", "decode", 1, "uniform", 131071, 131071, 6, page=16),
        # a decode step's queries over a bf16 cache
        case("weights_step_64", "weights", 64, "log", 128, 32768, 7, kv="bf16"),
        # the last 32 queries of each prompt observe the whole of it (4-bit cache)
        case("weights_observe_8", "weights", 8, "uniform", 4096, 16384, 8, q_len=32, page=16),
        # a few short odd sequences, head_dim 64
        case("weights_tiny", "weights", 3, "uniform", 65, 333, 9, heads=4, kv_heads=2, dim=64,
             page=16, kv="bf16", q_len=3, q_ragged=True),
        # prompts cut down to a budget after their prefill
        case("evict_prompts_32", "evict", 32, "uniform", 8192, 32768, 10, kv="bf16", budget=2048,
             first=4, recent=64),
        # running sequences that went one page over their budget
        case("evict_step_64", "evict", 64, "uniform", 1088, 1088, 11, kv="bf16", budget=1024,
             first=4, recent=32),
        # a few short sequences, one of them within the budget
        case("evict_tiny", "evict", 3, "uniform", 100, 400, 12, kv="bf16", dim=64, kv_heads=2,
             heads=4, page=16, budget=131, first=1, recent=17),
    ]


def _log_int(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["write", "decode", "weights", "evict"])
    dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 5, 8])
    c = dict(kind=kind, dim=dim, kv_heads=kv_heads, heads=kv_heads * group,
             page=rng.choice([16, 32, 64, 128]), layout=rng.choice(["NHD", "HND"]), window=0,
             strided=False, kv="mx4", q_len=1, q_ragged=False, budget=0, first=0, recent=0,
             lens=rng.choice(["log", "uniform"]), lens_seed=rng.randrange(1 << 20))
    if kind == "write":
        c["strided"] = rng.random() < 0.5
        if rng.random() < 0.4:                        # decode steps
            c.update(batch=_log_int(rng, 1, 256), lo=64, hi=_log_int(rng, 100, 8192),
                     q_len=rng.randint(1, 4))
        else:                                         # prompts
            hi = _log_int(rng, 33, 4096)
            c.update(batch=max(1, min(_log_int(rng, 1, 32), 16384 // hi)), lo=max(1, hi // 8),
                     hi=hi, q_len=hi, q_ragged=True)
    elif kind == "decode":
        hi = _log_int(rng, 40, 65536)
        c.update(batch=max(1, min(_log_int(rng, 1, 128), 1000000 // hi)), lo=max(8, hi // 16),
                 hi=hi, q_len=rng.randint(1, max(1, min(4, (32 if dim == 128 else 64) // group))),
                 q_ragged=rng.random() < 0.25,
                 window=rng.choice([0, 0, 0, _log_int(rng, 20, 4096)]))
    elif kind == "weights":
        hi = _log_int(rng, 70, 32768)
        c.update(batch=max(1, min(_log_int(rng, 1, 64), 200000 // hi)), lo=max(64, hi // 16),
                 hi=hi, q_len=rng.choice([1, 1, 2, 3, 8, 17, 32, 64]),
                 q_ragged=rng.random() < 0.25, kv=rng.choice(["bf16", "mx4"]))
    else:
        hi = _log_int(rng, 64, 32768)
        budget = _log_int(rng, 24, max(25, hi // 2))
        c.update(batch=max(1, min(_log_int(rng, 1, 64), 500000 // hi)), lo=max(16, hi // 4),
                 hi=hi, kv="bf16", budget=budget, first=rng.randint(0, min(8, budget // 4)),
                 recent=rng.randint(0, budget // 2))
    return c


def _lens(case):
    """(context lengths, query lengths) of a case; they follow from the case alone."""
    rng = random.Random(case["lens_seed"])
    lo, hi = case["lo"], case["hi"]
    f = _log_int if case["lens"] == "log" else (lambda r, a, b: r.randint(a, b))
    ctx = [f(rng, lo, hi) for _ in range(case["batch"])]
    if case["q_ragged"]:
        # prompts are new as a whole; shorter runs of new tokens vary from none up
        ql = [c if case["q_len"] >= hi else min(c, rng.randint(0, case["q_len"])) for c in ctx]
        if not any(ql):
            ql[0] = min(ctx[0], case["q_len"])
    else:
        ql = [min(c, case["q_len"]) for c in ctx]
    return ctx, ql


# ------------------------------------------------- the 4-bit microscaled form

def _block_exponent(x):
    """Biased power-of-two scale byte of each block of 32 (last axis): the
    exponent of the largest magnitude less that of the largest E2M1 value."""
    amax = x.abs().amax(-1)
    ex = torch.frexp(amax)[1]
    byte = (ex - 3).clamp(-127, 127) + 127
    byte = torch.where(amax > 0, byte, torch.zeros_like(byte))
    return torch.where(torch.isfinite(amax), byte, torch.full_like(byte, 255))


def _power(byte):
    """2^(byte - 127) in 32 bits; 255 stands for NaN."""
    b = byte.to(torch.int32)
    bits = torch.where(b == 0, torch.full_like(b, 0x00400000), b << 23)
    bits = torch.where(b == 255, torch.full_like(b, 0x7FC00000), bits)
    return bits.view(torch.float32)


def _quantise(x):
    """Rows [..., D] -> (two codes a byte [..., D/2], scale bytes [..., D/32])."""
    D = x.shape[-1]
    xb = x.float().reshape(*x.shape[:-1], D // 32, 32)
    byte = _block_exponent(xb)
    inv = _power((254 - byte).clamp(0, 254))
    y = xb * inv[..., None]
    a = y.abs()
    # round to nearest, ties to the even code; beyond 5 saturates to 6
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0))
    code = code + 8 * torch.signbit(y).to(torch.uint8)
    code = torch.where((byte == 255)[..., None], torch.zeros_like(code), code)
    code = code.reshape(*x.shape[:-1], D // 2, 2)
    return code[..., 0] + 16 * code[..., 1], byte.to(torch.uint8)


def _dequantise(codes, scales):
    """Codes [..., D/2] and scale bytes [..., D/32] -> values [..., D] in 32 bits."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    pair = torch.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1, 32)
    v = lut[pair.int()] * _power(scales)[..., None]
    return v.reshape(*codes.shape[:-1], -1)


# ------------------------------------------------------------------ prepare

def _pages(case, ctx, g, extra=0):
    """Block table [B, most pages] (-1 = unused) over a shuffled pool, and the pool's size."""
    ps = case["page"]
    need = [(c + ps - 1) // ps for c in ctx]
    total = sum(need) + extra + 3
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    n = torch.tensor(need, device="cuda")
    start = torch.cumsum(n, 0) - n
    j = torch.arange(max(need), device="cuda")
    at = (start[:, None] + j[None]).clamp(max=total - 1)
    table = torch.where(j[None] < n[:, None], perm[at], torch.full_like(perm[at], -1))
    return table.contiguous(), perm[sum(need):], total


def _cache_shape(case, pages, last):
    if case["layout"] == "NHD":
        return (pages, case["page"], case["kv_heads"], last)
    return (pages, case["kv_heads"], case["page"], last)


def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _quantised_cache(case, pages, g):
    """A 4-bit cache of random rows, filled some pages at a time."""
    D = case["dim"]
    codes = torch.empty(_cache_shape(case, pages, D // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty(_cache_shape(case, pages, D // 32), dtype=torch.uint8, device="cuda")
    # channels of unequal size, as keys and values have them
    channel = torch.exp(0.5 * torch.randn(D, generator=g, device="cuda"))
    step = max(1, (1 << 25) // (case["page"] * case["kv_heads"] * D))
    for p in range(0, pages, step):
        shape = _cache_shape(case, min(step, pages - p), D)
        c, s = _quantise(_randn(shape, g).float() * channel)
        codes[p:p + step], scales[p:p + step] = c, s
    return codes, scales


def _slots(case, table, ctx_t, most):
    """(page, slot, valid), each [B, most], of every token."""
    j = torch.arange(most, device="cuda")
    page = table.long()[:, (j // case["page"]).clamp(max=table.shape[1] - 1)]
    valid = j[None] < ctx_t[:, None]
    return torch.where(valid, page, torch.zeros_like(page)), (j % case["page"]).expand_as(page), valid


def _rows(case, cache, page, slot):
    """Cache rows of tokens (page, slot) [B, n] -> [B, Hkv, n, last]."""
    if case["layout"] == "NHD":
        return cache[page, slot].transpose(1, 2)
    h = torch.arange(case["kv_heads"], device="cuda")
    return cache[page[:, None, :], h[None, :, None], slot[:, None, :]]


def _q_rows(case, ctx_t, ql_t, mq):
    """(token index [B, mq], position [B, mq], valid [B, mq]) of the queries."""
    i = torch.arange(mq, device="cuda")
    start = torch.cumsum(ql_t, 0) - ql_t
    valid = i[None] < ql_t[:, None]
    tok = torch.where(valid, start[:, None] + i[None], torch.zeros_like(start[:, None] + i[None]))
    return tok, (ctx_t - ql_t)[:, None] + i[None], valid


def _scores(s, keys):
    """Scaled scores [B, Hkv, G, mq, L] in 32 bits, -inf where a query does not see a key."""
    c = s["case"]
    B, Hkv, G, D = c["batch"], c["kv_heads"], c["heads"] // c["kv_heads"], c["dim"]
    tok, pos, valid = _q_rows(c, s["ctx"].long(), s["ql"].long(), s["mq"])
    q = s["q"].float()[tok].reshape(B, s["mq"], Hkv, G, D).permute(0, 2, 3, 1, 4)
    L = keys.shape[2]
    x = torch.matmul(q.reshape(B, Hkv, G * s["mq"], D), keys.transpose(2, 3)) * s["scale"]
    x = x.reshape(B, Hkv, G, s["mq"], L)
    j = torch.arange(L, device="cuda")
    see = valid[:, :, None] & (j[None, None] <= pos[:, :, None])
    if c["window"] > 0:
        see = see & (j[None, None] > pos[:, :, None] - c["window"])
    return torch.where(see[:, None, None], x, torch.full_like(x, -math.inf)), tok, valid


def _plain_keys(s, cache, scales, page, slot, valid):
    rows = _rows(s["case"], cache, page, slot)
    v = rows.float() if scales is None else _dequantise(rows, _rows(s["case"], scales, page, slot))
    return torch.where(valid[:, None, :, None], v, torch.zeros_like(v))


def _plain_attention(s, with_out):
    c = s["case"]
    page, slot, valid = _slots(c, s["table"], s["ctx"], max(s["ctx_list"]))
    keys = _plain_keys(s, s["k"], s["ks"], page, slot, valid)
    x, tok, qv = _scores(s, keys)
    del keys
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    lse = (torch.exp(x - m).sum(-1).log() + m[..., 0])
    B, Hkv, G, mq = lse.shape
    flat = tok[qv]
    lse_out = torch.empty((s["total_q"], c["heads"]), device="cuda")
    lse_out[flat] = lse.permute(0, 3, 1, 2).reshape(B, mq, Hkv * G)[qv]
    if not with_out:
        return None, lse_out
    p = torch.exp(x - m)
    den = p.sum(-1, keepdim=True)
    p = p / torch.where(den > 0, den, torch.ones_like(den))
    del x
    vals = _plain_keys(s, s["v"], s["vs"], page, slot, valid)
    o = torch.matmul(p.reshape(B, Hkv, G * mq, -1), vals).reshape(B, Hkv, G, mq, c["dim"])
    out = torch.empty((s["total_q"], c["heads"], c["dim"]), device="cuda", dtype=torch.bfloat16)
    out[flat] = o.permute(0, 3, 1, 2, 4).reshape(B, mq, Hkv * G, c["dim"])[qv].to(torch.bfloat16)
    return out, lse_out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    ctx, ql = _lens(case)
    s = dict(case=dict(case), ctx_list=ctx, ql_list=ql, mq=max(ql), total_q=sum(ql),
             scale=1.0 / math.sqrt(case["dim"]))
    s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    s["ql"] = torch.tensor(ql, dtype=torch.int32, device="cuda")
    D, Hkv, ps, kind = case["dim"], case["kv_heads"], case["page"], case["kind"]
    keep = -(-case["budget"] // ps) if kind == "evict" else 0
    s["table"], spare, s["pages"] = _pages(case, ctx, g, extra=case["batch"] * keep)
    if kind == "write":
        width = Hkv * D * (case["heads"] // Hkv + 2) if case["strided"] else 2 * Hkv * D
        fused = _randn((s["total_q"], width), g)
        s["k_new"] = fused[:, -2 * Hkv * D:-Hkv * D].unflatten(1, (Hkv, D))
        s["v_new"] = fused[:, -Hkv * D:].unflatten(1, (Hkv, D))
        for n in "kv":
            s[n] = torch.zeros(_cache_shape(case, s["pages"], D // 2), dtype=torch.uint8, device="cuda")
            s[n + "s"] = torch.zeros(_cache_shape(case, s["pages"], D // 32), dtype=torch.uint8,
                                     device="cuda")
        # the bf16 pages that the rows are read back into: the new tokens' alone
        s["back_table"], _, back = _pages(case, ctx, g)
        s["k_out"] = torch.zeros(_cache_shape(case, back, D), dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.zeros_like(s["k_out"])
    elif case["kv"] == "bf16":
        s["k"], s["v"] = (_randn(_cache_shape(case, s["pages"], D), g) for _ in "kv")
        s["ks"] = s["vs"] = None
    else:
        s["k"], s["ks"] = _quantised_cache(case, s["pages"], g)
        s["v"], s["vs"] = _quantised_cache(case, s["pages"], g) if kind == "decode" else (None, None)
    if kind in ("decode", "weights"):
        s["q"] = _randn((s["total_q"], case["heads"], D), g)
    if kind == "weights":
        s["lse"] = _plain_attention(s, False)[1]
    if kind in ("weights", "evict"):
        u = torch.rand((s["pages"], Hkv, ps), generator=g, device="cuda")
        # running totals: a few keys hold most of the weight; exact repeats occur
        s["total"] = torch.floor(256 * u / (1.001 - u)) / 4096
    if kind == "evict":
        rows = torch.arange(case["batch"] * keep, device="cuda").reshape(case["batch"], keep)
        s["dst_table"] = spare[:case["batch"] * keep][rows].contiguous()
        s["kept"] = torch.full((case["batch"], Hkv, case["budget"]), -1, dtype=torch.int32,
                               device="cuda")
        s["new_ctx"] = torch.zeros(case["batch"], dtype=torch.int32, device="cuda")
    if own:
        from paged_attention_gb300 import binding as B
        s["p"] = B.PaProblem(
            num_seqs=case["batch"], num_q_heads=case["heads"], num_kv_heads=Hkv, head_dim=D,
            page_size=ps, num_pages=s["pages"], max_pages_per_seq=s["table"].shape[1],
            total_q_tokens=s["total_q"], max_q_len=s["mq"], max_context_len=max(ctx),
            layout=B.PA_NHD if case["layout"] == "NHD" else B.PA_HND,
            kv_dtype=B.PA_BF16 if case["kv"] == "bf16" else B.PA_MX4, sm_scale=s["scale"],
            window=case["window"])
        s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if kind == "write":
            s["back_pages"] = s["k_out"].shape[0]
        if kind == "decode":
            s["ws"] = torch.zeros(B.pa_mx4_workspace_size(s["p"]), dtype=torch.uint8, device="cuda")
            s["out"] = torch.empty((s["total_q"], case["heads"], D), dtype=torch.bfloat16,
                                   device="cuda")
            s["lse_out"] = torch.empty((s["total_q"], case["heads"]), device="cuda")
    return s


# ---------------------------------------------------------------------- run

def _put(case, cache, page, slot, rows):
    """Rows [n, Hkv, last] to tokens (page, slot) [n]."""
    if case["layout"] == "NHD":
        cache[page, slot] = rows
    else:
        cache[page, :, slot] = rows


def _new_tokens(s, table):
    """(page, slot) of every new token, in the order of the rows."""
    ql, ctx = s["ql"].long(), s["ctx"].long()
    b = torch.repeat_interleave(torch.arange(len(s["ql_list"]), device="cuda"), ql,
                                output_size=s["total_q"])
    i = torch.arange(s["total_q"], device="cuda") - (torch.cumsum(ql, 0) - ql)[b]
    pos = (ctx - ql)[b] + i
    return table.long()[b, pos // s["case"]["page"]], pos % s["case"]["page"]


def _run_write(s):
    c = s["case"]
    if own:
        from paged_attention_gb300 import binding as B
        B.pa_kv_append(s["p"], s["k_new"], s["v_new"], s["table"], s["ctx"], s["ql"], s["k"],
                       s["ks"], s["v"], s["vs"], None, s["err"])
        B.pa_kv_expand(s["p"], s["k"], s["ks"], s["v"], s["vs"], s["table"], s["ctx"], s["ql"],
                       s["back_table"], s["back_pages"], s["k_out"], s["v_out"], s["err"])
    else:
        page, slot = _new_tokens(s, s["table"])
        to_page, to_slot = _new_tokens(s, s["back_table"])
        codes, scales = _quantise(torch.stack((s["k_new"], s["v_new"])))
        _put(c, s["k"], page, slot, codes[0])
        _put(c, s["v"], page, slot, codes[1])
        _put(c, s["ks"], page, slot, scales[0])
        _put(c, s["vs"], page, slot, scales[1])
        back = _dequantise(codes, scales).to(torch.bfloat16)
        _put(c, s["k_out"], to_page, to_slot, back[0])
        _put(c, s["v_out"], to_page, to_slot, back[1])
    return {"k": s["k_out"], "v": s["v_out"]}


def _run_decode(s):
    if own:
        from paged_attention_gb300 import binding as B
        B.pa_decode_mx4(s["p"], s["q"], s["k"], s["ks"], s["v"], s["vs"], s["table"], s["ctx"],
                        s["ql"], s["ws"], s["out"], s["lse_out"])
        return {"out": s["out"], "lse": s["lse_out"]}
    out, lse = _plain_attention(s, True)
    return {"out": out, "lse": lse}


def _run_weights(s):
    c = s["case"]
    if own:
        from paged_attention_gb300 import binding as B
        B.pa_key_weights(s["p"], s["q"], s["k"], s["ks"], s["table"], s["ctx"], s["ql"], s["lse"],
                         s["total"], s["err"])
        return {"total": s["total"]}
    page, slot, valid = _slots(c, s["table"], s["ctx"], max(s["ctx_list"]))
    x, tok, _ = _scores(s, _plain_keys(s, s["k"], s["ks"], page, slot, valid))
    B_, Hkv, G = c["batch"], c["kv_heads"], c["heads"] // c["kv_heads"]
    lse = s["lse"][tok].reshape(B_, s["mq"], Hkv, G).permute(0, 2, 3, 1)
    w = torch.exp(x - lse[..., None]).sum((2, 3))                       # [B, Hkv, L]
    b, j = torch.nonzero(valid, as_tuple=True)
    s["total"][page[b, j], :, slot[b, j]] += w[b, :, j]
    return {"total": s["total"]}


def _run_evict(s):
    c = s["case"]
    if own:
        from paged_attention_gb300 import binding as B
        B.pa_kv_evict(s["p"], c["budget"], c["first"], c["recent"], s["k"], None, s["v"], None,
                      s["total"], s["table"], s["dst_table"], s["ctx"], s["kept"], s["new_ctx"],
                      s["err"])
        return {n: s[n] for n in ("k", "v", "total", "kept", "new_ctx")}
    budget, ctx = c["budget"], s["ctx"].long()
    most = max(max(s["ctx_list"]), budget)
    page, slot, valid = _slots(c, s["table"], ctx, most)
    h = torch.arange(c["kv_heads"], device="cuda")
    total = s["total"][page[:, None], h[None, :, None], slot[:, None]]  # [B, Hkv, L]
    j = torch.arange(most, device="cuda")
    safe = (j[None] < c["first"]) | (j[None] >= ctx[:, None] - c["recent"])
    key = torch.where(safe[:, None], torch.full_like(total, math.inf), total)
    key = torch.where(valid[:, None], key, torch.full_like(total, -math.inf))
    order = torch.sort(key, dim=-1, descending=True, stable=True)[1][..., :budget]
    kept = torch.sort(order, -1)[0]
    over = ctx > budget
    s["kept"][over] = kept[over].int()
    s["new_ctx"].copy_(torch.minimum(ctx, torch.full_like(ctx, budget)))
    b, hh, i = torch.nonzero(over[:, None, None].expand(-1, c["kv_heads"], budget), as_tuple=True)
    src = kept[b, hh, i]
    ps = c["page"]
    sp, ss = s["table"].long()[b, src // ps], src % ps
    dp, ds = s["dst_table"].long()[b, i // ps], i % ps
    for n in "kv":
        if c["layout"] == "NHD":
            s[n][dp, ds, hh] = s[n][sp, ss, hh]
        else:
            s[n][dp, hh, ds] = s[n][sp, hh, ss]
    s["total"][dp, hh, ds] = s["total"][sp, hh, ss]
    return {n: s[n] for n in ("k", "v", "total", "kept", "new_ctx")}


def run(state):
    return {"write": _run_write, "decode": _run_decode, "weights": _run_weights,
            "evict": _run_evict}[state["case"]["kind"]](state)


# --------------------------------------------------------------------- work

def work(case):
    ctx, ql = _lens(case)
    D, Hkv, H = case["dim"], case["kv_heads"], case["heads"]
    row = D * 2 if case["kv"] == "bf16" else D // 2 + D // 32     # a K (or V) row in the cache
    kind = case["kind"]
    if kind == "write":
        # new rows in, codes and scales out, bf16 rows out
        return {"bytes": sum(ql) * Hkv * 2 * (2 * D + row + 2 * D), "flops": 0}
    lo = [max(0, c - q - case["window"] + 1) if case["window"] else 0 for c, q in zip(ctx, ql)]
    keys = sum(c - a for c, a, q in zip(ctx, lo, ql) if q)
    pairs = 0
    for c, q in zip(ctx, ql):
        for i in range(q):
            p = c - q + i + 1
            pairs += min(p, case["window"]) if case["window"] else p
    if kind == "decode":
        rows = sum(ql) * H
        return {"bytes": keys * Hkv * 2 * row + rows * (4 * D + 4), "flops": 4 * D * H * pairs}
    if kind == "weights":
        return {"bytes": keys * Hkv * (row + 8) + sum(ql) * H * (2 * D + 4),
                "flops": 2 * D * H * pairs}
    over = [c for c in ctx if c > case["budget"]]
    kept = len(over) * case["budget"] * Hkv
    # every total of an evicted sequence in; kept rows and totals in and out; the kept lists out
    return {"bytes": sum(over) * Hkv * 4 + kept * (2 * 2 * row + 4 + 4), "flops": 0}


# -------------------------------------------------------------------- exact

def _exact_rows(case, cache, scales, table, n):
    """K or V rows [n, Hkv, D] of one sequence, in 64 bits."""
    ps, Hkv, D = case["page"], case["kv_heads"], case["dim"]
    pages = table[:-(-n // ps)].long()

    def dense(t):
        x = t[pages]
        if case["layout"] != "NHD":
            x = x.permute(0, 2, 1, 3)
        return x.reshape(-1, Hkv, t.shape[-1])[:n]

    x = dense(cache)
    if scales is None:
        return x.double()
    value = torch.empty((n, Hkv, D), dtype=torch.float64, device="cuda")
    for half in range(2):
        nib = (x >> (4 * half)) & 15
        mag, exp = (nib & 1).double(), ((nib >> 1) & 3).double()
        v = torch.where(exp == 0, mag * 0.5, (1 + mag / 2) * 2.0 ** (exp - 1))
        value[..., half::2] = torch.where(nib >= 8, -v, v)
    e = dense(scales).double()
    f = torch.where(e == 255, torch.full_like(e, math.nan), 2.0 ** (e - 127))
    return value * f.repeat_interleave(32, -1)


def _exact_scores(s, b, first, keys):
    """Scores [H, q, n] of sequence b, whose queries start at row `first`, in 64 bits."""
    c = s["case"]
    n, ql = s["ctx_list"][b], s["ql_list"][b]
    q = s["q"][first:first + ql].double().transpose(0, 1)              # [H, q, D]
    kh = keys.transpose(0, 1).repeat_interleave(c["heads"] // c["kv_heads"], 0)
    x = torch.bmm(q, kh.transpose(1, 2)) / math.sqrt(c["dim"])
    p = torch.arange(n - ql, n, device="cuda")[:, None]
    j = torch.arange(n, device="cuda")[None]
    hide = j > p
    if c["window"]:
        hide = hide | (j <= p - c["window"])
    return x.masked_fill(hide[None], -math.inf)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    kind = case["kind"]
    if kind == "evict":
        return None          # rows are moved, nothing is computed
    if kind == "write":
        got = {}
        for n, new, back in (("k", s["k_new"], s["k_out"]), ("v", s["v_new"], s["v_out"])):
            x = new.double().reshape(s["total_q"], c["kv_heads"], -1, 32)
            top = x.abs().amax(-1, keepdim=True)
            unit = 2.0 ** (torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top)))) - 2)
            z = x / unit
            grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
            far = (z.abs().clamp(max=6.0)[..., None] - grid).abs()
            near = far.amin(-1, keepdim=True)
            # of two equally near values the one with the even code
            even = torch.tensor([0, 1] * 4, dtype=torch.float64, device="cuda")
            pick = torch.where(far == near, even, torch.full_like(far, 2.0)).argmin(-1)
            y = torch.sign(z) * grid[pick] * unit
            out = back.double()
            at = 0
            for b, (n_ctx, ql) in enumerate(zip(s["ctx_list"], s["ql_list"])):
                pos = torch.arange(n_ctx - ql, n_ctx, device="cuda")
                page, slot = s["back_table"][b].long()[pos // c["page"]], pos % c["page"]
                rows = y[at:at + ql].reshape(ql, c["kv_heads"], -1)
                if c["layout"] == "NHD":
                    out[page, slot] = rows
                else:
                    out[page, :, slot] = rows
                at += ql
            got[n] = out
        return got
    if kind == "decode":
        out = torch.zeros((s["total_q"], c["heads"], c["dim"]), dtype=torch.float64, device="cuda")
        lse = torch.zeros((s["total_q"], c["heads"]), dtype=torch.float64, device="cuda")
    else:
        out, lse = s["total"].double(), None
    at = 0
    for b, (n, ql) in enumerate(zip(s["ctx_list"], s["ql_list"])):
        if ql:
            x = _exact_scores(s, b, at, _exact_rows(c, s["k"], s["ks"], s["table"][b], n))
            if kind == "decode":
                values = _exact_rows(c, s["v"], s["vs"], s["table"][b], n).transpose(0, 1)
                values = values.repeat_interleave(c["heads"] // c["kv_heads"], 0)
                out[at:at + ql] = torch.bmm(torch.softmax(x, -1), values).transpose(0, 1)
                lse[at:at + ql] = torch.logsumexp(x, -1).transpose(0, 1)
            else:
                w = torch.exp(x - s["lse"][at:at + ql].double().t()[..., None])
                w = w.reshape(c["kv_heads"], -1, n).sum(1)               # [Hkv, n]
                pos = torch.arange(n, device="cuda")
                out[s["table"][b].long()[pos // c["page"]], :, pos % c["page"]] += w.t()
            at += ql
    return {"out": out, "lse": lse} if kind == "decode" else {"total": out}
