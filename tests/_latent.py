"""Plain 64-bit forms of the latent-attention operators, for the GPU tests, and the
error bounds that the number formats give.

Attention goes request by request and token by token over the keys that a token
sees, so what stands elsewhere cannot enter.
"""
import math

import torch

from _step import HALF

LATENT, ROPE, NOPE, VALUE = 512, 64, 128, 128
EPS = 2.0 ** -24


def rows_ref(q, K, V, scale, dt):
    """One token: q [H, dk], K [keys, H or 1, dk], V [keys, H or 1, dv], in fp64 -> (o, lse, bound on o, bound on lse).

    A score is a sum of dk products, each exact to one rounding, in some order: off by at most
    dk + 4 roundings of the sum of magnitudes (scale and the factor log2(e) among the four).  The weight
    2^(s - m) then carries |s| + |m| roundings of its argument, 2 more of exp2, and the sum over n keys
    n of the norm; in bf16 the weights are rounded once more (half a step of bf16) for the second
    product but not in the norm.  The output is rounded to its type."""
    H = q.shape[0]
    n, dk = K.shape[0], q.shape[1]
    if n == 0:
        dv = V.shape[2]
        return (torch.zeros(H, dv, dtype=torch.float64), torch.full((H,), -math.inf, dtype=torch.float64),
                torch.full((H, dv), 1e-30, dtype=torch.float64), torch.zeros(H, dtype=torch.float64))
    K, V = K.expand(n, H, dk), V.expand(n, H, V.shape[2])
    s = scale * torch.einsum("hd,khd->hk", q, K)
    mag = scale * torch.einsum("hd,khd->hk", q.abs(), K.abs()).amax(1)
    w = torch.softmax(s, 1)
    o, lse = torch.einsum("hk,khd->hd", w, V), torch.logsumexp(s, 1)
    absum = torch.einsum("hk,khd->hd", w, V.abs())
    ds = (dk + 4) * EPS * mag + 4 * EPS * s.abs().amax(1) + (n + 16) * EPS
    bl = 2 * ds + 4 * EPS * lse.abs() + 1e-6
    rel = 2 * ds + (HALF[dt] if dt == torch.bfloat16 else 0)
    bo = absum * rel[:, None] * 1.01 + HALF[dt] * o.abs() * 1.01 + 1e-30
    return o, lse, bo, bl


def absorbed_ref(q, cache, table, cu, seq, scale):
    """(o, lse, bounds) of kda_latent_attention on the CPU; rows of q behind the last request: bound inf."""
    T, H, _ = q.shape
    n_pages, page, _ = cache.shape
    o = torch.zeros(T, H, LATENT, dtype=torch.float64)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64)
    bo, bl = torch.full_like(o, math.inf), torch.full_like(lse, math.inf)
    for n in range(table.shape[0]):
        lo, m, end = int(cu[n]), int(cu[n + 1]) - int(cu[n]), int(seq[n])
        keys = min(end, table.shape[1] * page)
        ids = table[n].long().repeat_interleave(page)[:keys]
        exists = (ids >= 0) & (ids < n_pages)
        rows = cache[ids.clamp(0, n_pages - 1), torch.arange(keys) % page].double()
        for i in range(m):
            p = end - m + i
            sel = torch.nonzero(exists[:max(0, min(p + 1, keys))])[:, 0]
            K = rows[sel][:, None]
            o[lo + i], lse[lo + i], bo[lo + i], bl[lo + i] = rows_ref(q[lo + i].double(), K, K[..., :LATENT], scale, q.dtype)
    return o, lse, bo, bl


def expanded_ref(q, k_nope, k_rope, v, cu, cu_k, scale, causal):
    """(o, lse, bounds) of kda_expanded_attention on the CPU; rows of q behind the last request: bound inf."""
    T, H, _ = q.shape
    o = torch.zeros(T, H, VALUE, dtype=torch.float64)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64)
    bo, bl = torch.full_like(o, math.inf), torch.full_like(lse, math.inf)
    for n in range(len(cu) - 1):
        lo, m = int(cu[n]), int(cu[n + 1]) - int(cu[n])
        a, b = int(cu_k[n]), int(cu_k[n + 1])
        K = torch.cat([k_nope[a:b], k_rope[a:b, None].expand(b - a, H, ROPE)], 2).double()
        V = v[a:b].double()
        for i in range(m):
            sees = max(0, b - a - m + i + 1) if causal else b - a
            o[lo + i], lse[lo + i], bo[lo + i], bl[lo + i] = rows_ref(q[lo + i].double(), K[:sees], V[:sees], scale, q.dtype)
    return o, lse, bo, bl


def turned(x, positions, inv_freq, factor, interleaved):
    """x [T, H, d] with its first 2 len(inv_freq) channels turned, fp64, and the bound on a kernel's error.

    A cosine or sine is off by at most an eighth of a turn's rounding (pi / 4 2^-24), the
    function's own 2 roundings and one of the factor: 5 roundings of the factor; the two products and
    their sum, 3 roundings of |a| + |b| times the factor; then the output's."""
    half = inv_freq.numel()
    out, bound = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    a, b = x[..., first].double(), x[..., second].double()
    w = positions.double()[:, None, None] * inv_freq.double()
    out[..., first] = factor * (a * w.cos() - b * w.sin())
    out[..., second] = factor * (b * w.cos() + a * w.sin())
    bound[..., first] = bound[..., second] = 8 * EPS * abs(factor) * (a.abs() + b.abs())
    bound[..., :2 * half] += HALF[x.dtype] * out[..., :2 * half].abs() * 1.01 + 1e-30
    return out, bound


def assert_close(got, ref, bound, what):
    got = got.double().cpu()
    live = torch.isfinite(bound)
    bad = live & ~((got - ref).abs() <= bound)
    bad &= ~(torch.isinf(ref) & (got == ref))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {int(live.sum())} out of bounds, worst "
                           f"{float(((got - ref).abs() / bound)[bad].max())} at {torch.nonzero(bad)[0].tolist()}")
