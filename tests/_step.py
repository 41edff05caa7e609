"""Plain 64-bit forms of the serving-step operators, for the GPU tests, and the
error bounds that the number formats give.

Everything here goes request by request and row by row over the keys that a row
sees, so what stands elsewhere cannot enter.
"""
import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}      # half a step, relative


def lay_out(lens, page, n_extra, gen, blocks=None):
    """Pages of requests with (cached, new) tokens each: block table [N, blocks], cu, seq, pages in the pool."""
    need = [max(0, -(-(a + b) // page)) for a, b in lens]
    blocks = max(1, max(need)) if blocks is None else blocks
    n_pages = sum(need) + n_extra
    order = torch.randperm(n_pages, generator=gen).tolist()
    table = torch.full((len(lens), blocks), -1, dtype=torch.int32)
    for n, k in enumerate(need):
        for b in range(k):
            table[n, b] = order.pop()
    cu = torch.tensor([0] + [b for _, b in lens]).cumsum(0).to(torch.int32)
    seq = torch.tensor([max(0, a + b) for a, b in lens], dtype=torch.int32)
    return table, cu, seq, n_pages


def attention_ref(q, k_cache, v_cache, table, cu, seq, scale, window):
    """(o, lse, bound on |o - o_kernel|, bound on lse) in fp64 on the CPU; q [T, Hq, d] and the
    caches are the stored values.  The bounds count, per row: the rounding of each product
    sum of d terms in fp32, of the weights to the storage type (bf16 only), of the sums over
    the keys in fp32, and of the output."""
    T, Hq, d = q.shape
    n_pages, Hkv, page, _ = k_cache.shape
    G = Hq // Hkv
    dt = q.dtype
    o = torch.zeros(T, Hq, d, dtype=torch.float64)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    bo, bl = torch.zeros_like(o), torch.zeros_like(lse)
    eps = 2.0 ** -24
    for n in range(table.shape[0]):
        lo, hi = int(cu[n]), int(cu[n + 1])
        m, end = hi - lo, int(seq[n])
        keys = min(end, table.shape[1] * page)
        ids = table[n].long().repeat_interleave(page)[:keys]
        exists = (ids >= 0) & (ids < n_pages)
        place = torch.arange(keys) % page
        at = ids.clamp(0, max(0, n_pages - 1))
        for i in range(m):
            p = end - m + i
            first = max(0, p - window + 1) if window > 0 else 0
            sel = torch.arange(first, min(p + 1, keys)) if p >= first else torch.arange(0)
            sel = sel[exists[sel]] if len(sel) else sel
            if len(sel) == 0:
                continue
            K = k_cache[at[sel], :, place[sel]].double().repeat_interleave(G, 1)     # [keys, Hq, d]
            V = v_cache[at[sel], :, place[sel]].double().repeat_interleave(G, 1)
            x = q[lo + i].double()
            s = scale * torch.einsum("hd,khd->hk", x, K)
            mag = scale * torch.einsum("hd,khd->hk", x.abs(), K.abs()).amax(1)
            w = torch.softmax(s, 1)
            lse[lo + i] = torch.logsumexp(s, 1)
            o[lo + i] = torch.einsum("hk,khd->hd", w, V)
            absum = torch.einsum("hk,khd->hd", w, V.abs())
            # a score is off by (d + 3) roundings of its magnitude; the running reference m, up to 8 octaves
            # above nothing, costs |s| roundings more in s - m; exp2 and the sums over the keys follow
            ds = (d + 4) * eps * mag + 4 * eps * s.abs().amax(1) + (len(sel) + 16) * eps
            bl[lo + i] = 2 * ds + 4 * eps * lse[lo + i].abs() + 1e-6
            rel = 2 * ds + (HALF[dt] if dt == torch.bfloat16 else 0)
            bo[lo + i] = absum * rel[:, None] * 1.01 + HALF[dt] * o[lo + i].abs() + 1e-30
    return o, lse, bo, bl


def tables_ref(ctx, new, free, table, page, n_tokens):
    """(table, cu, seq, slots, positions, taken), plain Python."""
    table = [list(r) for r in table]
    cu, seq, slots, pos, taken = [0], [], [], [], 0
    for n in range(len(ctx)):
        c, a = max(ctx[n], 0), max(new[n], 0)
        blocks = len(table[n])
        for b in range(min(-(-c // page), blocks), min(-(-(c + a) // page), blocks)):
            table[n][b] = free[taken] if taken < len(free) else -1
            taken += 1
        for p in range(c, c + a):
            b = p // page
            slots.append(table[n][b] * page + p % page if b < blocks and table[n][b] >= 0 else -1)
            pos.append(p)
        cu.append(cu[-1] + a)
        seq.append(c + a)
    slots = (slots + [-1] * n_tokens)[:n_tokens]
    pos = (pos + [0] * n_tokens)[:n_tokens]
    return table, cu, seq, slots, pos, taken


def verify_ref(target, draft, tokens, uniforms, lens):
    """(tokens, commit_len) with exact rational sums (Python integers over 2^-149 steps)."""
    from fractions import Fraction
    n, k1, V = target.shape
    out, commit = [], []
    frac = lambda x: Fraction(x) if x > 0 else Fraction(0)  # noqa: E731  (NaN compares false)
    for i in range(n):
        a = 0
        while a < lens[i]:
            x = int(tokens[i, a])
            if not 0 <= x < V:
                break
            q = 1.0 if draft is None else float(draft[i, a, x])
            p = float(target[i, a, x])
            if not (math.isfinite(q) and math.isfinite(p) and Fraction(float(uniforms[i, a])) * Fraction(q) < Fraction(p)):
                break
            a += 1
        row = [frac(float(x)) for x in target[i, a]]
        left = row
        if a < lens[i]:
            if draft is None:
                left = [Fraction(0) if v == int(tokens[i, a]) else r for v, r in enumerate(row)]
            else:
                left = [max(r - frac(float(x)), Fraction(0)) for r, x in zip(row, draft[i, a])]
            if sum(left) == 0:
                left = row
        total, u = sum(left), Fraction(float(uniforms[i, k1 - 1]))
        drawn, acc = None, Fraction(0)
        for v, r in enumerate(left):
            acc += r
            if acc > u * total:
                drawn = v
                break
        if drawn is None:
            positive = [v for v, r in enumerate(left) if r > 0]
            drawn = positive[-1] if positive else V - 1
        out.append([int(x) for x in tokens[i, :a]] + [drawn] + [-1] * (k1 - 1 - a))
        commit.append(a + 1)
    return out, commit
