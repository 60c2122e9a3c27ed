"""Plain 64-bit forms of the operators of a serving step (include/pa_step.h), on
the CPU, written from the definitions; sizes in the tests are small."""
import math

import torch

NHD, HND = 0, 1
PAD = (-1, 0, -1)


def up(a, b):
    return -(-a // b)


def take(seq_lens, q_lens, table, stack, count, *, page, pages, rows, max_q, max_ctx):
    """(table, context_lens, [(row_seq, position, slot)], pages left, error bits)."""
    table = [list(r) for r in table]
    ctx, maps, err, free, at = [], [PAD] * rows, 0, max(0, min(count, pages)), 0
    err = 0 if free == count else 1
    out_of_pages = False
    for b, (n, q) in enumerate(zip(seq_lens, q_lens)):
        cut = max(0, min(q, max_q))
        row0, at = at, at + cut
        if n < 0 or q < 0 or q > max_q or n + q > max_ctx or at > rows:
            err |= 1
            ctx.append(max(0, min(n, max_ctx)))
            continue
        need = up(n + q, page) - up(n, page)
        if need and (out_of_pages or need > free):
            out_of_pages = True
            err |= 16
            ctx.append(n)
            continue
        for j in range(need):
            table[b][up(n, page) + j] = stack[free - 1 - j]
        free -= need
        ctx.append(n + q)
        for i in range(q):
            p = n + i
            pg = table[b][p // page]
            if not 0 <= pg < pages:
                err |= 2
            maps[row0 + i] = (b, p, pg * page + p % page if 0 <= pg < pages else -1)
    return table, ctx, maps, free, err


def give_back(seq_lens, keep_lens, table, stack, count, *, page, pages, max_ctx):
    """(stack, pages on it, error bits)."""
    stack, err = list(stack), 0 if 0 <= count <= pages else 1
    count = max(0, min(count, pages))
    for b, (n, k) in enumerate(zip(seq_lens, keep_lens)):
        if k < 0 or k > n or n > max_ctx:
            err |= 1
            continue
        for j in range(up(k, page), up(n, page)):
            if count >= pages:
                err |= 1
                continue
            ok = 0 <= table[b][j] < pages
            err |= 0 if ok else 2
            stack[count] = table[b][j] if ok else -1
            count += 1
    return stack, count, err


def rotate(x, positions, inv_freq, rot, interleaved, factor):
    """x [T, heads, D] turned, in 64 bits; and what its rounding errors go by."""
    x = x.double()
    out, size = x.clone(), torch.zeros_like(x)
    half = rot // 2
    angle = positions.double()[:, None] * inv_freq.double()[None]
    cos, sin = torch.cos(angle)[:, None] * factor, torch.sin(angle)[:, None] * factor
    i = torch.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    u, v = x[..., a], x[..., b]
    out[..., a], out[..., b] = u * cos - v * sin, v * cos + u * sin
    size[..., a] = size[..., b] = (u.abs() + v.abs()) * abs(factor)
    return out, size


def exponent(top):
    """Least e in [-50, 50] with top <= 127 * 2^e."""
    if not math.isfinite(top):
        return 50
    e = -50
    while e < 50 and top > 127.0 * 2.0 ** e:
        e += 1
    return e


def bounds(k):
    """k [n, D] of one page and head -> (int8 [2, D], scale)."""
    k = k.double()
    fine = torch.where(torch.isnan(k), torch.full_like(k, math.inf), k)
    e = exponent(float(fine.abs().max()))
    hi = torch.ceil(k.amax(0) / 2.0 ** e).clamp(-127, 127)
    lo = torch.floor(k.amin(0) / 2.0 ** e).clamp(-127, 127)
    nan = torch.isnan(k).any(0)
    hi, lo = torch.where(nan, 127.0, hi), torch.where(nan, -127.0, lo)
    return torch.stack((hi, lo)).to(torch.int8), 2.0 ** e


def seen_pages(pos, page, window):
    """First and number of the pages that a query at pos sees a key of."""
    first = max(0, pos - window + 1) // page if window else 0
    return first, pos // page + 1 - first


def select(q, bnd, scale, table_row, pos, *, budget, num_first, num_recent, page, pages, window):
    """q [G, D] of one row and KV head, bnd [pages, 2, D], scale [pages] -> list of pages."""
    first, n = seen_pages(pos, page, window)
    if n <= budget:
        got = list(range(first, first + n))
        return got + [-1] * (budget - n)
    codes, power = [], []
    for row in q.double():
        mag = torch.where(torch.isnan(row), torch.zeros_like(row), row.abs())
        e = exponent(float(mag.max()))
        c = torch.round(row / 2.0 ** e).clamp(-127, 127)
        codes.append(torch.where(torch.isnan(row), torch.zeros_like(c), c))
        power.append(2.0 ** e)
    score = []
    for j in range(n):
        if j < num_first or j >= n - num_recent:
            score.append(math.inf)
            continue
        pg = table_row[first + j]
        if not 0 <= pg < pages:
            score.append(-math.inf)
            continue
        hi, lo = bnd[pg].double()
        # (where the largest is no less than the smallest, max(c * hi, c * lo) is the same)
        score.append(max(p * float((c * torch.where(c > 0, hi, lo)).sum())
                         for c, p in zip(codes, power)) * float(scale[pg]))
    order = sorted(range(n), key=lambda j: (-score[j], j))[:budget]
    return [first + j for j in sorted(order)]


def attend(q, k, v, positions_of_keys, pos, window, scale):
    """q [G, D]; k, v [n, D] (listed keys) -> out, lse, weighted sizes, largest score size."""
    q, k, v = q.double(), k.double(), v.double()
    at = torch.as_tensor(positions_of_keys)
    see = at <= pos
    if window:
        see &= at > pos - window
    k, v = k[see], v[see]
    G, D = q.shape
    if k.shape[0] == 0:
        z = torch.zeros((G, D), dtype=torch.float64)
        return z, torch.full((G,), -math.inf, dtype=torch.float64), z, torch.zeros(G)
    x = q @ k.t() * scale
    size = (q.abs() @ k.abs().t()).amax(-1) * scale
    w = torch.softmax(x, -1)
    return w @ v, torch.logsumexp(x, -1), w @ v.abs(), size
