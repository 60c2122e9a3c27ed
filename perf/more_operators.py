"""Measured cases of the operators of a serving step around attention: what a
step needs besides attending to the whole of a paged K/V cache.

Five paths, each the calls a user's program makes:

  pages    pages of finished requests go back to a free stack, and the new
           tokens of the step's requests get theirs: block table, lengths, and
           per new token its sequence, position and slot in the cache
  rope     rotary positions on the queries and keys of the new tokens, the
           queries into a dense tensor, keys and values into the cache
  bounds   per page and KV head, each channel's smallest and largest key in 8
           bits, of the pages that got new tokens
  select   per new token and KV head, the pages with the highest bound on a
           logit, with the first and the newest ones
  attend   attention of the new tokens over the pages selected for them

Lengths come from the case (``lens``, ``lo``, ``hi``, ``lens_seed``), values
from the seed.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------- cases

def listed():
    base = dict(heads=32, kv_heads=8, dim=128, page=64, layout="NHD", window=0, strided=True,
                q_len=1, q_ragged=False, pad=0, done=0.0, budget=0, first=1, recent=2, rot=128,
                inter=False, scaling="none", far=0)

    def case(name, kind, batch, lens, lo, hi, lens_seed, **kw):
        c = dict(base, name=name, kind=kind, batch=batch, lens=lens, lo=lo, hi=hi,
                 lens_seed=lens_seed)
        c.update(kw)
        return c

    return [
        # one decode step of 64 running requests, two of which drafts were taken back from
        case("pages_step_64", "pages", 64, "log", 128, 32768, 1, done=0.03, pad=8),
        # prompts that come in where finished requests left, 16-token pages
        case("pages_prompts_256", "pages", 256, "log", 17, 4096, 2, q_len=4096, q_ragged=True,
             page=16, done=0.5, pad=5),
        # a decode step's rows out of a fused QKV projection: latency
        case("rope_step_64", "rope", 64, "log", 128, 32768, 3),
        # a batch of long prompts' chunks at far positions: interleaved pairs, half of the
        # head, scaled frequencies, 16-token pages
        case("rope_chunks_far", "rope", 16, "uniform", 257, 2048, 4, q_len=2048, q_ragged=True,
             page=16, layout="HND", rot=64, inter=True, scaling="yarn", far=100000),
        # the last page of every running request after a decode step
        case("bounds_step_64", "bounds", 64, "log", 128, 32768, 5),
        # all pages of new prompts
        case("bounds_prompts_8", "bounds", 8, "uniform", 4096, 16384, 6, q_len=16384,
             q_ragged=True, layout="HND"),
        # a decode step's choice of 32 pages of 64 tokens
        case("select_step_64", "select", 64, "log", 128, 32768, 7, budget=32),
        # one very long sequence in small pages
        case("select_long_1", "select", 1, "uniform", 131071, 131071, 8, page=16, budget=256),
        # the smallest attention: a few short sequences, head_dim 64
        case("attend_tiny", "attend", 3, "uniform", 37, 300, 9, heads=4, kv_heads=1, dim=64,
             page=16, budget=5),
        # an ordinary decode step over 32 pages of 64 tokens
        case("attend_step_64", "attend", 64, "log", 128, 32768, 10, budget=32),
        # the largest batch: long contexts, 64 heads, two draft tokens
        case("attend_drafts_128", "attend", 128, "uniform", 1024, 16384, 11, heads=64, q_len=3,
             layout="HND", budget=40),
        # one very long sequence in small pages
        case("attend_long_1", "attend", 1, "uniform", 131071, 131071, 12, page=16, budget=256),
    ]


def _log_int(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["pages", "rope", "bounds", "select", "attend", "attend"])
    dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 5, 7, 8, 16])
    page = rng.choice([16, 32, 64, 128, 256])
    c = dict(kind=kind, dim=dim, kv_heads=kv_heads, heads=kv_heads * group, page=page,
             layout=rng.choice(["NHD", "HND"]), window=0, strided=rng.random() < 0.7, q_len=1,
             q_ragged=False, pad=rng.choice([0, 0, 3, 8]), done=0.0, budget=0, first=1, recent=2,
             rot=dim, inter=rng.random() < 0.4, scaling="none", far=0,
             lens=rng.choice(["log", "uniform"]), lens_seed=rng.randrange(1 << 20))
    if kind in ("pages", "rope", "bounds"):
        if rng.random() < 0.4:                        # decode steps
            c.update(batch=_log_int(rng, 1, 256), lo=64, hi=_log_int(rng, 100, 8192),
                     q_len=rng.randint(1, 4))
        else:                                         # prompts
            hi = _log_int(rng, 33, 4096)
            c.update(batch=max(1, min(_log_int(rng, 1, 64), 16384 // hi)), lo=max(1, hi // 8),
                     hi=hi, q_len=hi, q_ragged=True)
        c["done"] = rng.choice([0.0, 0.1, 0.6])
        c["rot"] = rng.choice([dim, dim, dim // 2, 16, dim - 16])
        c["scaling"] = rng.choice(["none", "none", "linear", "ntk", "yarn", "bands"])
        c["far"] = rng.choice([0, 0, _log_int(rng, 1000, 1000000)])
    else:
        hi = _log_int(rng, 40, 65536)
        q_len = rng.randint(1, 4)
        batch = min(_log_int(rng, 1, 128), 300000 // hi, 24000 // (q_len * c["heads"]))
        c.update(batch=max(1, batch), lo=max(8, hi // 16), hi=hi, q_len=q_len,
                 q_ragged=rng.random() < 0.25, budget=_log_int(rng, 1, max(2, 2560 // page)),
                 window=rng.choice([0, 0, 0, _log_int(rng, 20, 4096)]))
        c["first"] = rng.randint(0, c["budget"] // 3)
        c["recent"] = rng.randint(0, c["budget"] // 2)
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


def _left(case):
    """Per request of the step before: (tokens it held, tokens that stay)."""
    rng = random.Random(case["lens_seed"] + 1)
    f = _log_int if case["lens"] == "log" else (lambda r, a, b: r.randint(a, b))
    held = [f(rng, case["lo"], case["hi"]) for _ in range(case["batch"])]
    keep = []
    for n in held:
        u = rng.random()
        # finished, or up to three drafts taken back, or as it was
        keep.append(0 if u < case["done"] else max(0, n - rng.randint(1, 3)) if u > 0.8 else n)
    return held, keep


def _up(a, b):
    return -(-a // b)


# ----------------------------------------------------------- rotary positions

def _frequencies(rot, scaling):
    """(inverse frequencies [rot / 2], factor on cos and sin)."""
    base, factor, old = 500000.0, 8.0, 8192.0
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        return [x / factor for x in f], 1.0
    if scaling == "yarn":
        at = lambda turns: rot * math.log(old / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(0.0, math.floor(at(32.0))), min(rot - 1.0, math.ceil(at(1.0)))
        hi = hi if hi != lo else hi + 0.001
        ramp = [min(1.0, max(0.0, (i - lo) / (hi - lo))) for i in range(rot // 2)]
        return [x / factor * r + x * (1 - r) for x, r in zip(f, ramp)], 0.1 * math.log(factor) + 1
    if scaling == "bands":
        out = []
        for x in f:
            wave = 2 * math.pi / x
            mix = min(1.0, max(0.0, (old / wave - 1.0) / (4.0 - 1.0)))
            out.append(x / factor * (1 - mix) + x * mix)
        return out, 1.0
    return f, 1.0


# ------------------------------------------------------------------ prepare

def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _cache_shape(case, pages):
    if case["layout"] == "NHD":
        return (pages, case["page"], case["kv_heads"], case["dim"])
    return (pages, case["kv_heads"], case["page"], case["dim"])


def _table(need, perm, width):
    """Block table [B, width] (-1 = unused): the first need[b] entries of row b out of perm."""
    n = torch.tensor(need, device="cuda")
    start = torch.cumsum(n, 0) - n
    j = torch.arange(width, device="cuda")
    at = (start[:, None] + j[None]).clamp(max=perm.numel() - 1)
    return torch.where(j[None] < n[:, None], perm[at], torch.full_like(perm[at], -1)).contiguous()


def _rows(ctx, ql, total):
    """(sequence, position) of every new token; -1 and 0 in the rows behind the last."""
    ql, ctx = torch.tensor(ql, device="cuda"), torch.tensor(ctx, device="cuda")
    seq = torch.full((total,), -1, dtype=torch.int32, device="cuda")
    pos = torch.zeros(total, dtype=torch.int32, device="cuda")
    b = torch.repeat_interleave(torch.arange(len(ql), device="cuda"), ql)
    i = torch.arange(b.numel(), device="cuda") - (torch.cumsum(ql, 0) - ql)[b]
    seq[:b.numel()] = b.int()
    pos[:b.numel()] = ((ctx - ql)[b] + i).int()
    return seq, pos


def _two_power(amax):
    """Least e in [-50, 50] with amax <= 127 * 2^e."""
    m, ex = torch.frexp(amax)
    e = torch.where(m <= 127.0 / 128.0, ex - 7, ex - 6)
    e = torch.where(amax > 0, e, torch.full_like(e, -50))
    return e.clamp(-50, 50)


def _bound_codes(lo, hi):
    """Channels' smallest and largest values [..., D] (fp32) -> (int8 [..., 2, D]: largest
    rounded up, smallest rounded down; fp32 scale [...])."""
    e = _two_power(torch.maximum(lo.abs(), hi.abs()).amax(-1))
    s = torch.ldexp(torch.ones_like(lo[..., 0]), e)
    up = torch.ceil(hi / s[..., None]).clamp(-127, 127)
    down = torch.floor(lo / s[..., None]).clamp(-127, 127)
    return torch.stack((up, down), -2).to(torch.int8), s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    ctx, ql = _lens(case)
    D, Hkv, ps, kind, B = case["dim"], case["kv_heads"], case["page"], case["kind"], case["batch"]
    total = sum(ql) + case["pad"]
    s = dict(case=dict(case), ctx_list=ctx, ql_list=ql, total=total, scale=1.0 / math.sqrt(D))
    need = [_up(c, ps) for c in ctx]
    width = max(need)
    pages = sum(need) + 3
    if kind == "pages":
        held, keep = _left(case)
        old = [c - q for c, q in zip(ctx, ql)]
        have, was = [_up(n, ps) for n in old], [_up(n, ps) for n in held]
        # requests that stay keep their pages in the new table; the free ones are below
        take = sum(need) - sum(have)
        pages = sum(was) + sum(have) + take + 7
        perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        s["most_old"] = max(max(held), max(ql))
        s["old_table"] = _table(was, perm, _up(s["most_old"], ps))
        s["table"] = _table(have, perm[sum(was):], width)
        s["free"] = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
        spare = perm[sum(was) + sum(have):]
        s["free"][:spare.numel()] = spare
        s["count"] = torch.tensor([spare.numel()], dtype=torch.int32, device="cuda")
        for n, v in (("held", held), ("keep", keep), ("old", old), ("ql", ql)):
            s[n] = torch.tensor(v, dtype=torch.int32, device="cuda")
        s["between"], s["left"] = torch.zeros_like(s["count"]), torch.zeros_like(s["count"])
        s["ctx"] = torch.zeros_like(s["old"])
        s["seq"], s["pos"], s["slots"] = (torch.zeros(total, dtype=torch.int32, device="cuda")
                                          for _ in range(3))
        s["most"] = max(ctx)
    else:
        s["seq"], s["pos"] = _rows(ctx, ql, total)
        s["most"] = max(ctx)
        valid = s["seq"] >= 0
        if kind in ("rope", "bounds"):
            # pages of the new tokens alone: from the one of the first new token on
            at = [(c - q) // ps for c, q in zip(ctx, ql)]
            need = [n - a if q else 0 for n, a, q in zip(need, at, ql)]
            pages = sum(need) + 3
            perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
            table = _table(need, perm, max(need))
            b, p = s["seq"].long().clamp(min=0), s["pos"].long()
            page = table[b, (p // ps - torch.tensor(at, device="cuda")[b]).clamp(min=0)].long()
            s["slots"] = torch.where(valid, page * ps + p % ps, torch.full_like(p, -1)).int()
        else:
            perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
            s["table"] = _table(need, perm, width)
    if kind == "rope":
        s["pos"] = torch.where(valid, s["pos"] + case["far"], s["pos"])
        s["most"] += case["far"]
        H = case["heads"]
        if case["strided"]:
            fused = _randn((total, (H + 2 * Hkv) * D), g)
            parts = fused.split([H * D, Hkv * D, Hkv * D], 1)
        else:
            parts = [_randn((total, n * D), g) for n in (H, Hkv, Hkv)]
        s["q"], s["k_new"], s["v_new"] = (x.unflatten(1, (-1, D)) for x in parts)
        s["q_out"] = torch.zeros((total, H, D), dtype=torch.bfloat16, device="cuda")
        s["k"], s["v"] = (torch.zeros(_cache_shape(case, pages), dtype=torch.bfloat16,
                                      device="cuda") for _ in "kv")
        f, s["factor"] = _frequencies(case["rot"], case["scaling"])
        s["freq"] = torch.tensor(f, dtype=torch.float64, device="cuda")
    if kind == "bounds":
        s["k"] = _randn(_cache_shape(case, pages), g)
        s["bounds"] = torch.zeros((pages, Hkv, 2, D), dtype=torch.int8, device="cuda")
        s["bound_scale"] = torch.zeros((pages, Hkv), device="cuda")
    if kind in ("select", "attend"):
        s["q"] = _randn((total, case["heads"], D), g)
        s["selected"] = torch.full((total, Hkv, case["budget"]), -1, dtype=torch.int32,
                                   device="cuda")
    if kind == "select":
        # channels of unequal size and place, as keys have them
        mid = torch.randn((pages, Hkv, D), generator=g, device="cuda") * 0.5
        half = 2.4 + 0.3 * torch.randn((pages, Hkv, D), generator=g, device="cuda")
        size = torch.exp(0.5 * torch.randn((Hkv, D), generator=g, device="cuda"))
        lo, hi = ((x * size).to(torch.bfloat16).float() for x in (mid - half, mid + half))
        s["bounds"], s["bound_scale"] = _bound_codes(torch.minimum(lo, hi), torch.maximum(lo, hi))
    if kind == "attend":
        s["k"], s["v"] = (_randn(_cache_shape(case, pages), g) for _ in "kv")
        # lists as a selection leaves them; the queries of a sequence share what they
        # choose by score
        rank = torch.rand((B, Hkv, width), generator=g, device="cuda")
        s["selected"] = _top_pages(s, rank[s["seq"].long().clamp(min=0)])
    if own:
        from paged_attention_gb300 import binding as A
        s["p"] = A.PaProblem(
            num_seqs=B, num_q_heads=case["heads"], num_kv_heads=Hkv, head_dim=D, page_size=ps,
            num_pages=pages, max_pages_per_seq=max(width, _up(s["most"], ps)) if kind == "rope"
            else width, total_q_tokens=total, max_q_len=max(ql), max_context_len=s["most"],
            layout=A.PA_NHD if case["layout"] == "NHD" else A.PA_HND, kv_dtype=A.PA_BF16,
            sm_scale=s["scale"], window=case["window"])
        s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if kind == "pages":
            s["p_old"] = A.PaProblem.from_buffer_copy(s["p"])
            s["p_old"].max_context_len = s["most_old"]
            s["p_old"].max_pages_per_seq = s["old_table"].shape[1]
        if kind == "rope":
            scaling = A.PaRopeScaling(
                kind=getattr(A, "PA_ROPE_" + case["scaling"].upper()), rotary_dim=case["rot"],
                base=500000.0, factor=8.0, original_context=8192.0,
                high_turns=4.0 if case["scaling"] == "bands" else 32.0, low_turns=1.0)
            freq, factor = A.pa_rope_inv_freq(scaling)
            s["steps"] = A.pa_rope_steps(freq).cuda()
            s["rope"] = A.PaRope(rotary_dim=case["rot"], interleaved=int(case["inter"]),
                                 cos_sin_scale=factor)
        if kind == "attend":
            s["ws"] = torch.zeros(A.pa_selected_workspace_size(s["p"], case["budget"]),
                                  dtype=torch.uint8, device="cuda")
            s["out"] = torch.zeros((total, case["heads"], D), dtype=torch.bfloat16, device="cuda")
            s["lse"] = torch.zeros((total, case["heads"]), device="cuda")
    return s


# ---------------------------------------------------------------------- run

def _spans(first, last):
    """(row, index) of the pairs first[r] <= index < last[r], row by row."""
    n = (last - first).clamp(min=0)
    r = torch.repeat_interleave(torch.arange(n.numel(), device="cuda"), n)
    return r, torch.arange(r.numel(), device="cuda") - (torch.cumsum(n, 0) - n)[r] + first[r]


def _run_pages(s):
    c, ps = s["case"], s["case"]["page"]
    if own:
        from paged_attention_gb300 import binding as A
        A.pa_pages_return(s["p_old"], s["held"], s["keep"], s["old_table"], s["free"], s["count"],
                          s["between"], s["err"])
        A.pa_pages_take(s["p"], s["old"], s["ql"], s["table"], s["free"], s["between"], s["ctx"],
                        s["seq"], s["pos"], s["slots"], s["left"], s["err"])
    else:
        held, keep, old, ql = (s[n].long() for n in ("held", "keep", "old", "ql"))
        b, j = _spans((keep + ps - 1) // ps, (held + ps - 1) // ps)
        at = s["count"].long() + torch.arange(b.numel(), device="cuda")
        s["free"][at] = s["old_table"][b, j]
        s["between"].copy_(s["count"] + b.numel())
        ctx = old + ql
        b, j = _spans((old + ps - 1) // ps, (ctx + ps - 1) // ps)
        at = s["between"].long() - 1 - torch.arange(b.numel(), device="cuda")
        s["table"][b, j] = s["free"][at]
        s["left"].copy_(s["between"] - b.numel())
        s["ctx"].copy_(ctx)
        b, p = _spans(old, ctx)
        n = b.numel()
        s["seq"].fill_(-1)
        s["pos"].fill_(0)
        s["slots"].fill_(-1)
        s["seq"][:n], s["pos"][:n] = b.int(), p.int()
        s["slots"][:n] = (s["table"][b, p // ps].long() * ps + p % ps).int()
    return {"free": s["free"], "table": s["table"], "ctx": s["ctx"], "seq": s["seq"],
            "pos": s["pos"], "slots": s["slots"], "left": s["left"]}


def _rotate(case, x, cos, sin):
    """x [T, heads, D] in 32 bits, its first ``rot`` elements turned."""
    rot = case["rot"]
    a, rest = x[..., :rot], x[..., rot:]
    if case["inter"]:
        u, v = a[..., 0::2], a[..., 1::2]
        a = torch.stack((u * cos - v * sin, v * cos + u * sin), -1).flatten(-2)
    else:
        u, v = a[..., :rot // 2], a[..., rot // 2:]
        a = torch.cat((u * cos - v * sin, v * cos + u * sin), -1)
    return torch.cat((a, rest), -1)


def _put(case, cache, slots, rows):
    page, slot = slots // case["page"], slots % case["page"]
    if case["layout"] == "NHD":
        cache[page, slot] = rows
    else:
        cache[page, :, slot] = rows


def _run_rope(s):
    c = s["case"]
    if own:
        from paged_attention_gb300 import binding as A
        A.pa_rope_append(s["p"], s["rope"], s["steps"], s["q"], s["k_new"], s["v_new"], s["pos"],
                         s["slots"], s["q_out"], s["k"], None, s["v"], None, s["err"])
    else:
        angle = s["pos"].double()[:, None] * s["freq"][None]
        cos, sin = ((f(angle) * s["factor"]).float()[:, None] for f in (torch.cos, torch.sin))
        n = sum(s["ql_list"])
        s["q_out"][:n] = _rotate(c, s["q"].float(), cos, sin)[:n].to(torch.bfloat16)
        slots = s["slots"][:n].long()
        _put(c, s["k"], slots, _rotate(c, s["k_new"].float(), cos, sin)[:n].to(torch.bfloat16))
        _put(c, s["v"], slots, s["v_new"][:n])
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _run_bounds(s):
    c, ps = s["case"], s["case"]["page"]
    if own:
        from paged_attention_gb300 import binding as A
        A.pa_page_bounds(s["p"], s["k"], s["slots"], s["bounds"], s["bound_scale"], s["err"])
    else:
        slots = s["slots"][:sum(s["ql_list"])].long()
        page, used = slots // ps, slots % ps + 1
        last = torch.ones_like(page, dtype=torch.bool)
        last[:-1] = page[1:] != page[:-1]
        page, used = page[last], used[last]
        k = s["k"][page].float()                      # [n, slots, heads, D] or [n, heads, slots, D]
        at = torch.arange(ps, device="cuda")
        there = at[None] < used[:, None]
        there, axis = ((there[:, :, None, None], 1) if c["layout"] == "NHD"
                       else (there[:, None, :, None], 2))
        lo = torch.where(there, k, torch.full_like(k, math.inf)).amin(axis)
        hi = torch.where(there, k, torch.full_like(k, -math.inf)).amax(axis)
        s["bounds"][page], s["bound_scale"][page] = _bound_codes(lo, hi)
    return {"bounds": s["bounds"], "scale": s["bound_scale"]}


def _seen(s):
    """(first, number) of the pages that each row's query sees any key of."""
    c, p = s["case"], s["pos"].long()
    first = torch.zeros_like(p)
    if c["window"]:
        first = (p - c["window"] + 1).clamp(min=0) // c["page"]
    n = p // c["page"] + 1 - first
    return first, torch.where(s["seq"] >= 0, n, torch.zeros_like(n))


def _top_pages(s, score):
    """Of scores [T, Hkv, pages] the budget's page numbers, ascending, -1 behind them."""
    c, budget = s["case"], s["case"]["budget"]
    first, n = (x[:, None, None] for x in _seen(s))
    j = torch.arange(score.shape[-1], device="cuda")[None, None] - first
    kept = (j < c["first"]) | (j >= n - c["recent"])
    key = torch.where(kept, torch.full_like(score, math.inf), score)
    key = torch.where((j >= 0) & (j < n), key, torch.full_like(key, -math.inf))
    order = torch.sort(key, dim=-1, descending=True, stable=True)[1][..., :budget]
    many = torch.full_like(order, 1 << 40)
    got = torch.where(torch.arange(order.shape[-1], device="cuda") < n, order, many).sort(-1)[0]
    out = torch.full((*score.shape[:2], budget), -1, dtype=torch.int32, device="cuda")
    out[..., :got.shape[-1]] = torch.where(got == many, torch.full_like(got, -1), got).int()
    return out


def _run_select(s):
    c = s["case"]
    if own:
        from paged_attention_gb300 import binding as A
        A.pa_select_pages(s["p"], c["budget"], c["first"], c["recent"], s["q"], s["bounds"],
                          s["bound_scale"], s["table"], s["seq"], s["pos"], s["selected"],
                          s["err"])
        return {"selected": s["selected"]}
    Hkv, G, D = c["kv_heads"], c["heads"] // c["kv_heads"], c["dim"]
    q = s["q"].float().reshape(s["total"], Hkv, G, D)
    e = _two_power(q.abs().amax(-1))
    qs = torch.ldexp(torch.ones_like(q[..., 0]), e)
    code = torch.round(q / qs[..., None]).clamp(-127, 127)
    # a product with the larger of two codes is one with the upper where q is positive
    both = torch.cat((code.clamp(min=0), code.clamp(max=0)), -1)          # [T, Hkv, G, 2 D]
    table = s["table"].long().clamp(min=0)
    score = torch.empty((s["total"], Hkv, table.shape[1]), device="cuda")
    seq = s["seq"].long().clamp(min=0)
    step = max(1, (1 << 28) // (table.shape[1] * Hkv * 2 * D))
    for t in range(0, s["total"], step):
        page = table[seq[t:t + step]]                                     # [t, pages]
        b = s["bounds"][page].float().flatten(-2).permute(0, 2, 3, 1)     # [t, Hkv, 2 D, pages]
        dot = torch.matmul(both[t:t + step], b)                           # whole numbers
        dot = (dot * qs[t:t + step, :, :, None]).amax(2)
        score[t:t + step] = dot * s["bound_scale"][page].transpose(1, 2)
    n = sum(s["ql_list"])
    s["selected"][:n] = _top_pages(s, score)[:n]
    return {"selected": s["selected"]}


def _run_attend(s):
    c = s["case"]
    if own:
        from paged_attention_gb300 import binding as A
        A.pa_decode_selected(s["p"], c["budget"], s["q"], s["k"], s["v"], s["table"], s["seq"],
                             s["pos"], s["selected"], s["ws"], s["out"], s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    Hkv, G, D, ps = c["kv_heads"], c["heads"] // c["kv_heads"], c["dim"], c["page"]
    T = s["total"]
    out = torch.zeros((T, c["heads"], D), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((T, c["heads"]), device="cuda")
    h = torch.arange(Hkv, device="cuda")[None, :, None, None]
    slot = torch.arange(ps, device="cuda")[None, None, None]
    n = sum(s["ql_list"])
    step = max(1, (1 << 28) // (Hkv * c["budget"] * ps * D))
    for t in range(0, n, step):
        z = min(n, t + step)
        sel = s["selected"][t:z].long()
        page = s["table"][s["seq"][t:z].long()[:, None, None], sel.clamp(min=0)].long()[..., None]
        at = (page, slot, h) if c["layout"] == "NHD" else (page, h, slot)
        key = (sel[..., None] * ps + slot).flatten(2)                     # positions
        p = s["pos"][t:z].long()[:, None, None]
        see = (sel[..., None] >= 0).expand(-1, -1, -1, ps).flatten(2) & (key <= p)
        if c["window"]:
            see = see & (key > p - c["window"])
        q = s["q"][t:z].float().reshape(z - t, Hkv, G, D)
        k = s["k"][at].flatten(2, 3).float()
        x = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
        x = torch.where(see[:, :, None], x, torch.full_like(x, -math.inf))
        m = x.amax(-1, keepdim=True)
        w = torch.exp(x - torch.where(torch.isfinite(m), m, torch.zeros_like(m)))
        den = w.sum(-1, keepdim=True)
        v = s["v"][at].flatten(2, 3).float()
        o = torch.matmul(w, v) / torch.where(den > 0, den, torch.ones_like(den))
        out[t:z] = o.reshape(z - t, -1, D).to(torch.bfloat16)
        lse[t:z] = (den.log() + m).reshape(z - t, -1)
    return {"out": out, "lse": lse}


def run(state):
    return {"pages": _run_pages, "rope": _run_rope, "bounds": _run_bounds, "select": _run_select,
            "attend": _run_attend}[state["case"]["kind"]](state)


# --------------------------------------------------------------------- work

def work(case):
    ctx, ql = _lens(case)
    D, Hkv, H, ps, kind = case["dim"], case["kv_heads"], case["heads"], case["page"], case["kind"]
    rows = sum(ql)
    if kind == "pages":
        held, keep = _left(case)
        back = sum(_up(n, ps) - _up(k, ps) for n, k in zip(held, keep))
        new = sum(_up(c, ps) - _up(c - q, ps) for c, q in zip(ctx, ql))
        # lengths in, page numbers from one place to another, three maps and the lengths out
        return {"bytes": 20 * case["batch"] + 8 * (back + new) + 12 * (rows + case["pad"]),
                "flops": 0}
    if kind == "rope":
        pairs = rows * (H + Hkv) * case["rot"] // 2
        return {"bytes": rows * (2 * 2 * D * (H + 2 * Hkv) + 8), "flops": 6 * pairs}
    if kind == "bounds":
        pages = sum(_up(c, ps) - (c - q) // ps for c, q in zip(ctx, ql) if q)
        keys = sum(c - (c - q) // ps * ps for c, q in zip(ctx, ql) if q)
        return {"bytes": Hkv * (keys * 2 * D + pages * (2 * D + 4)) + 4 * rows,
                "flops": 2 * keys * Hkv * D}
    seen, taken, dots, keys = 0, 0, 0, 0
    for c, q in zip(ctx, ql):
        per = []
        for p in range(c - q, c):
            first = max(0, p - case["window"] + 1) // ps if case["window"] else 0
            per.append(p // ps + 1 - first)
            got = min(per[-1], case["budget"])
            dots += per[-1]
            # the page of the query itself ends at it (it is left out where a choice by
            # score alone does so)
            keys += got * ps - (ps - 1 - p % ps)
        seen += max(per, default=0)
        taken += min(max(per, default=0), case["budget"])
    lists = rows * Hkv * case["budget"] * 4
    if kind == "select":
        # the bounds of a sequence's pages once for all its queries
        return {"bytes": seen * (Hkv * (2 * D + 4) + 4) + rows * H * 2 * D + lists,
                "flops": 4 * D * H * dots}
    # the pages of a sequence's queries once: they share most of them
    return {"bytes": taken * ps * Hkv * 4 * D + rows * H * (4 * D + 4) + lists,
            "flops": 4 * D * H * keys}


# -------------------------------------------------------------------- exact

def exact(case, seed):
    kind = case["kind"]
    if kind == "pages":
        return None          # whole numbers that are moved, nothing is computed
    s = prepare(case, seed)
    c, ps, D, Hkv = s["case"], case["page"], case["dim"], case["kv_heads"]
    G = case["heads"] // Hkv
    n = sum(s["ql_list"])
    if kind == "rope":
        half = case["rot"] // 2
        f = s["freq"]
        got = {"q": s["q_out"].double(), "k": s["k"].double(), "v": s["v"].double()}
        slots = s["slots"][:n].long()
        i = torch.arange(half, device="cuda")
        first, second = (2 * i, 2 * i + 1) if case["inter"] else (i, i + half)
        turn = s["factor"] * torch.polar(torch.ones_like(f), s["pos"][:n].double()[:, None] * f)
        for name, x in (("q", s["q"]), ("k", s["k_new"])):
            y = x[:n].double().clone()
            z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
            y[..., first], y[..., second] = z.real, z.imag
            if name == "q":
                got["q"][:n] = y
            else:
                _put(c, got["k"], slots, y)
        _put(c, got["v"], slots, s["v_new"][:n].double())
        return got
    if kind == "bounds":
        codes, scale = s["bounds"].long(), s["bound_scale"].double()
        used = {x // ps: x % ps + 1 for x in s["slots"][:n].tolist()}    # the last one counts
        for page, m in used.items():
            k = s["k"][page].double()
            k = k[:m] if c["layout"] == "NHD" else k.transpose(0, 1)[:m]
            lo, hi = k.amin(0), k.amax(0)                                # [Hkv, D]
            top = torch.maximum(lo.abs(), hi.abs()).amax(-1) / 127
            unit = torch.exp2(torch.ceil(torch.log2(top)).clamp(-50, 50))
            codes[page, :, 0] = torch.ceil(hi / unit[:, None]).long()
            codes[page, :, 1] = torch.floor(lo / unit[:, None]).long()
            scale[page] = unit
        return {"bounds": codes, "scale": scale}
    first, many = _seen(s)
    if kind == "select":
        out = s["selected"].long()
        for t in range(n):
            b, lo, m = int(s["seq"][t]), int(first[t]), int(many[t])
            page = s["table"][b, lo:lo + m].long()
            q = s["q"][t].double()                                       # [H, D]
            top = q.abs().amax(-1) / 127
            eq = torch.ceil(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
            eq = torch.where(top > 0, eq, torch.full_like(eq, -50.0)).clamp(-50, 50)
            code = torch.round(q / torch.exp2(eq)[:, None])
            hi, low = (s["bounds"][page][:, :, i].double() for i in (0, 1))   # [m, Hkv, D]
            for h in range(Hkv):
                cq = code[h * G:(h + 1) * G]
                best = torch.maximum(cq[:, None] * hi[None, :, h], cq[:, None] * low[None, :, h])
                y = (best.sum(-1) * torch.exp2(eq[h * G:(h + 1) * G])[:, None]).amax(0)
                y = y * s["bound_scale"][page, h].double()
                y[:case["first"]] = math.inf
                y[max(0, m - case["recent"]):] = math.inf
                pick = torch.argsort(-y, stable=True)[:case["budget"]].sort()[0] + lo
                out[t, h] = -1
                out[t, h, :pick.numel()] = pick
        return {"selected": out}
    out = torch.zeros((s["total"], case["heads"], D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((s["total"], case["heads"]), dtype=torch.float64, device="cuda")
    slot = torch.arange(ps, device="cuda")
    for t in range(n):
        row = s["table"][int(s["seq"][t])].long()
        p = s["pos"][t].long()
        for h in range(Hkv):
            sel = s["selected"][t, h].long()
            sel = sel[sel >= 0]
            if c["layout"] == "NHD":
                k, v = (s[x][row[sel], :, h].reshape(-1, D).double() for x in "kv")
            else:
                k, v = (s[x][row[sel], h].reshape(-1, D).double() for x in "kv")
            at = (sel[:, None] * ps + slot).flatten()
            hide = at > p
            if case["window"]:
                hide = hide | (at <= p - case["window"])
            x = s["q"][t, h * G:(h + 1) * G].double() @ k.t() / math.sqrt(D)
            x = x.masked_fill(hide[None], -math.inf)
            lse[t, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
            w = torch.where(hide.all(), torch.zeros_like(x), torch.softmax(x, -1))
            out[t, h * G:(h + 1) * G] = w @ v
    return {"out": out, "lse": lse}
