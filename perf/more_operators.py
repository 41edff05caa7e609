"""Cases and plain forms of the latent-attention operators.

The softmax-attention layers of a model that mixes them with KDA layers may keep
one shared latent vector a token instead of keys and values of each head: a
latent of 512 channels, which serves all heads as their values, and a rotated
key part of 64 channels beside it.  ``rotary`` turns queries by their positions,
``append`` writes latents and turned key parts into the paged cache, ``absorbed``
attends over that cache from queries that hold the key projection already
(576 channels against the cache's rows), ``expanded`` attends over keys and
values that were projected from the latents again (192 and 128 channels a head),
as prompts do.

``listed()`` and ``draw()`` give cases, ``prepare()`` what a serving program
holds before a call, ``run()`` one pass through one operator: in plain torch
where ``own`` is false, through this package's entry points where it is true.
``exact()`` computes the same from the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
LATENT, ROPE, NOPE, VALUE = 512, 64, 128, 128              # channels: latent, rotated part, the rest of a key, a value
SCALE = (NOPE + ROPE) ** -0.5                              # of the scores, in both forms


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the rotated part of a decode step's queries, on its way into the absorbed queries' tail
        dict(name="rotary_decode", op="rotary", n=48, heads=32, dim=64, rot=64, gap=128, far=9000, interleaved=True,
             scaling=1.0, factor=1.0, dtype="bf16"),
        # a long prompt's queries, half of each head turned, frequencies stretched for a long context
        dict(name="rotary_prompt", op="rotary", n=20001, heads=32, dim=128, rot=64, gap=0, far=1000000, interleaved=False,
             scaling=8.0, factor=1.2079, dtype="bf16"),
        # one decode step of a mid-sized batch
        dict(name="latent_append_decode", op="append", n=96, page=16, pages=8192, far=9000, interleaved=True, rotated=True,
             dtype="bf16"),
        # the latents of a long prompt chunk
        dict(name="latent_append_prompt", op="append", n=40001, page=64, pages=1024, far=1000000, interleaved=False,
             rotated=True, dtype="bf16"),
        # a few short conversations, one token each
        dict(name="absorbed_decode_few", op="absorbed", n=4, ctx_lo=90, ctx_hi=1500, new_lo=1, new_hi=1, heads=32, page=16,
             dtype="bf16"),
        # a serving batch of decode requests: the cache's bytes count
        dict(name="absorbed_decode", op="absorbed", n=64, ctx_lo=1000, ctx_hi=16384, new_lo=1, new_hi=1, heads=32, page=64,
             dtype="bf16"),
        # many heads over long contexts, one token each: as many operations as bytes
        dict(name="absorbed_many_heads", op="absorbed", n=24, ctx_lo=2001, ctx_hi=32000, new_lo=1, new_hi=1, heads=128,
             page=64, dtype="bf16"),
        # verification of seven drafted tokens and the last one of each request
        dict(name="absorbed_verify", op="absorbed", n=32, ctx_lo=700, ctx_hi=8191, new_lo=8, new_hi=8, heads=32, page=32,
             dtype="bf16"),
        # a mixed step of a small model in single precision, odd head count
        dict(name="absorbed_fp32", op="absorbed", n=6, ctx_lo=17, ctx_hi=2100, new_lo=1, new_hi=9, heads=5, page=16,
             dtype="fp32"),
        # a prompt, causal
        dict(name="expanded_prompt", op="expanded", n=1, ctx_lo=0, ctx_hi=0, new_lo=8192, new_hi=8192, heads=32, causal=True,
             dtype="bf16"),
        # prompts of many lengths against an earlier part of their context, joined to the rest by the lse
        dict(name="expanded_context", op="expanded", n=12, ctx_lo=0, ctx_hi=2501, new_lo=1, new_hi=700, heads=16, causal=False,
             dtype="bf16"),
        # a few short prompts in single precision
        dict(name="expanded_fp32", op="expanded", n=5, ctx_lo=0, ctx_hi=600, new_lo=3, new_hi=260, heads=5, causal=True,
             dtype="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "append", "absorbed", "absorbed", "absorbed", "expanded", "expanded"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op == "rotary":
        dim = rng.choice([32, 64, 96, 128, 192, 256])
        return dict(op=op, n=_log(rng, 1, 20001 if dtype == "bf16" else 8000), heads=rng.choice([1, 2, 5, 8, 16, 32]), dim=dim,
                    rot=rng.choice([r for r in (16, 32, 64, 96, 128, 256) if r <= dim]), gap=rng.choice([0, 8, 128, 512]),
                    far=_log(rng, 10, 1000000), interleaved=rng.random() < 0.5, scaling=rng.choice([1.0, 4.0, 8.0]),
                    factor=rng.choice([1.0, 1.0693, 1.2079]), dtype=dtype)
    if op == "append":
        n, page = _log(rng, 1, 40001 if dtype == "bf16" else 20000), rng.choice([16, 32, 64, 128, 256])
        return dict(op=op, n=n, page=page, pages=_up(n, page) + rng.randint(8, 512), far=_log(rng, 10, 1000000),
                    interleaved=rng.random() < 0.5, rotated=rng.random() < 0.75, dtype=dtype)
    if op == "absorbed":
        kind = rng.choice(["decode", "verify", "chunk"])
        heads, page = rng.choice([1, 5, 8, 16, 20, 32, 40, 64, 96, 128]), rng.choice([16, 32, 64, 128, 256])
        wide = dtype == "bf16"
        if kind == "decode":
            return dict(op=op, n=_log(rng, 1, 64 if wide and heads <= 32 else 16), ctx_lo=rng.choice([0, 1, 300]),
                        ctx_hi=_log(rng, 301, 16384 if wide else 3000), new_lo=1, new_hi=1, heads=heads, page=page, dtype=dtype)
        heads = min(heads, 40)
        if kind == "verify":
            new = rng.randint(2, 16)
            return dict(op=op, n=_log(rng, 1, 16 if wide else 4), ctx_lo=rng.choice([0, 1, 300]),
                        ctx_hi=_log(rng, 301, 8192 if wide else 1500), new_lo=new, new_hi=new, heads=heads, page=page, dtype=dtype)
        return dict(op=op, n=rng.randint(1, 4), ctx_lo=0, ctx_hi=_log(rng, 64, 6000 if wide else 600), new_lo=rng.choice([0, 1, 17]),
                    new_hi=_log(rng, 64, 600 if wide else 130), heads=min(heads, 20), page=page, dtype=dtype)
    wide = dtype == "bf16"
    return dict(op=op, n=rng.randint(1, 8), ctx_lo=rng.choice([0, 1, 100]), ctx_hi=_log(rng, 101, 6000 if wide else 1000),
                new_lo=rng.choice([0, 1, 17]), new_hi=_log(rng, 18, 3000 if wide else 500), heads=rng.choice([1, 2, 5, 8, 16]),
                causal=rng.random() < 0.7, dtype=dtype)


def _spread(lo, hi, n):
    """n lengths from lo to hi, spread over their logarithm."""
    if n == 1:
        return [hi]
    a, b = math.log(lo + 1), math.log(hi + 1)
    return [int(round(math.exp(a + (b - a) * i / (n - 1)))) - 1 for i in range(n)]


def _lengths(case):
    """(earlier tokens, new tokens) of each request: the case's alone, in no particular order."""
    n = case["n"]
    ctx, new = _spread(case["ctx_lo"], case["ctx_hi"], n), _spread(case["new_lo"], case["new_hi"], n)
    step = next(s for s in range(n // 2 + 1, 2 * n + 2) if math.gcd(s, n) == 1)
    return [(ctx[i], new[(i * step) % n]) for i in range(n)]


def _up(a, b):
    return -(-a // b)


# ------------------------------------------------------------------ inputs
def _frequencies(rot, scaling):
    """Turns a position by theta ** (-2 i / rot); a longer context slows the slow half of them down."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    slow = torch.linspace(0.0, 1.0, rot // 2, dtype=torch.float64)
    return (f * (1.0 - slow) + f / scaling * slow).float().cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    state, dt = dict(case), DTYPES[case["dtype"]]
    rows = lambda *shape: torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(dt)  # noqa: E731
    if case["op"] == "rotary":
        n, heads, dim, gap = case["n"], case["heads"], case["dim"], case["gap"]
        state["x"] = rows(n, heads, gap + dim)[..., gap:]                       # a slice of the projection's output
        state["out"] = torch.empty(n, heads, dim, dtype=dt, device="cuda")
        state["positions"] = torch.randint(0, case["far"], (n,), generator=gen, device="cuda", dtype=torch.int32)
        state["inv_freq"] = _frequencies(case["rot"], case["scaling"])
        return state
    if case["op"] == "append":
        n, slots = case["n"], case["pages"] * case["page"]
        both = rows(n, LATENT + ROPE)                                           # one projection gives both parts
        state["c"], state["k_rope"] = both[:, :LATENT], both[:, LATENT:]
        state["cache"] = torch.zeros(case["pages"], case["page"], LATENT + ROPE, dtype=dt, device="cuda")
        state["slot_map"] = torch.randperm(slots, generator=gen, device="cuda")[:n].contiguous()
        if n > 8:
            state["slot_map"][-3:] = -1                                         # padding of a fixed-size step
        state["positions"] = torch.randint(0, case["far"], (n,), generator=gen, device="cuda", dtype=torch.int32)
        state["inv_freq"] = _frequencies(ROPE, 1.0)
        return state
    n, heads, lens = case["n"], case["heads"], _lengths(case)
    order = torch.randperm(n, generator=gen, device="cuda")
    pairs = torch.tensor(lens, dtype=torch.int32, device="cuda")[order]
    ctx, new = pairs[:, 0].contiguous(), pairs[:, 1].contiguous()
    total = sum(b for _, b in lens)
    state["max_new"] = max(b for _, b in lens)
    state["cu_seqlens"] = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    state["cu_seqlens"][1:] = torch.cumsum(new, 0)
    state["seq_len"] = (ctx + new).contiguous()
    if case["op"] == "absorbed":
        page = case["page"]
        n_pages = sum(_up(a + b, page) for a, b in lens) + 16
        blocks = max(1, max(_up(a + b, page) for a, b in lens))
        pages = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
        col, have = torch.arange(blocks, device="cuda")[None, :], (state["seq_len"] + page - 1) // page
        first = torch.cumsum(have, 0) - have
        table = torch.where(col < have[:, None], pages[(first[:, None] + col).clamp(max=n_pages - 1)], -1)
        state["block_table"] = table.to(torch.int32).contiguous()
        state["cache"] = rows(n_pages, page, LATENT + ROPE)
        state["q"] = rows(total, heads, LATENT + ROPE)
        return state
    keys = sum(a + b for a, b in lens)
    state["max_keys"] = max(a + b for a, b in lens)
    state["cu_seqlens_k"] = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    state["cu_seqlens_k"][1:] = torch.cumsum(state["seq_len"], 0)
    both = rows(keys, heads, NOPE + VALUE)                                      # one projection of the latents gives both
    state["k_nope"], state["v"] = both[..., :NOPE], both[..., NOPE:]
    state["k_rope"] = rows(keys, ROPE)
    state["q"] = rows(total, heads, NOPE + ROPE)
    return state


# ------------------------------------------------------------------ one pass
def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _own_rotary(s):
    import kimi_delta_attention_chunked_gb300 as kda
    return kda.kda_rotary(s["x"], s["positions"], s["inv_freq"], factor=s["factor"], interleaved=s["interleaved"], out=s["out"])


def _own_append(s):
    import kimi_delta_attention_chunked_gb300 as kda
    turn = dict(positions=s["positions"], inv_freq=s["inv_freq"], interleaved=s["interleaved"]) if s["rotated"] else {}
    kda.kda_latent_append(s["c"], s["k_rope"], s["cache"], s["slot_map"], **turn)
    return s["cache"]


def _own_absorbed(s):
    import kimi_delta_attention_chunked_gb300 as kda
    return kda.kda_latent_attention(s["q"], s["cache"], s["block_table"], s["cu_seqlens"], s["seq_len"], SCALE, want_lse=True)


def _own_expanded(s):
    import kimi_delta_attention_chunked_gb300 as kda
    return kda.kda_expanded_attention(s["q"], s["k_nope"], s["k_rope"], s["v"], s["cu_seqlens"], s["cu_seqlens_k"],
                                      scale=SCALE, causal=s["causal"], want_lse=True)


_own = {"rotary": _own_rotary, "append": _own_append, "absorbed": _own_absorbed, "expanded": _own_expanded}


def _turn(x, positions, inv_freq, factor, interleaved):
    """x [T, H, rot] turned by position * frequency: pairs (2 i, 2 i + 1), or (i, i + rot / 2)."""
    angle = positions.double()[:, None] * inv_freq.double()                     # 64 bits: positions reach a million
    cos, sin = (factor * angle.cos()).float()[:, None], (factor * angle.sin()).float()[:, None]
    half = inv_freq.numel()
    pairs = x.float().unflatten(-1, (half, 2)) if interleaved else x.float().unflatten(-1, (2, half)).transpose(-1, -2)
    a, b = pairs[..., 0], pairs[..., 1]
    both = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return (both if interleaved else both.transpose(-1, -2)).flatten(-2)


def _plain_rotary(s):
    """The first `rot` channels of each head are turned, the others copied."""
    x, rot, out = s["x"], s["rot"], s["out"]
    out[..., :rot] = _turn(x[..., :rot], s["positions"], s["inv_freq"], s["factor"], s["interleaved"]).to(out.dtype)
    out[..., rot:] = x[..., rot:]
    return out


def _plain_append(s):
    """Row t, latent and turned key part, goes to place slot % page of page slot // page; a negative slot is skipped."""
    cache, slot, page = s["cache"], s["slot_map"], s["page"]
    part = s["k_rope"]
    if s["rotated"]:
        part = _turn(part[:, None], s["positions"], s["inv_freq"], 1.0, s["interleaved"])[:, 0].to(part.dtype)
    live = slot >= 0
    at = torch.where(live, slot, slot.amax())               # a skipped row writes what the last slot's own row writes
    row = torch.where(live, torch.arange(slot.numel(), device=slot.device), slot.argmax())
    cache[at // page, at % page] = torch.cat([s["c"], part], dim=-1)[row]
    return cache


def _softmax(scores, seen):
    """Weights without their norm, the norm and the lse of rows of scores; rows that see nothing give zeros and -inf."""
    scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    weights = scores.sub_(top).exp_()
    norm = weights.sum(dim=-1, keepdim=True)
    return weights, norm, (top + torch.log(norm))[..., 0]


def _rows_of(s):
    """Request of each new token, its place there; and token rows of each request, padded."""
    cu, total = s["cu_seqlens"].long(), s["q"].shape[0]
    t = torch.arange(total, device=cu.device)
    r = torch.searchsorted(cu[1:], t, right=True)
    i = torch.arange(s["max_new"], device=cu.device)
    return r, t - cu[r], (cu[:-1, None] + i).clamp(max=max(0, total - 1)), i


def _plain_absorbed(s):
    """softmax(scale q c^T) c[:512] of each new token and head over the cache rows up to its own position."""
    q, table, seq = s["q"], s["block_table"], s["seq_len"].long()
    n, heads, most = s["n"], s["heads"], s["max_new"]
    new = (s["cu_seqlens"][1:] - s["cu_seqlens"][:-1]).long()
    r, at, index, i = _rows_of(s)
    keys = s["cache"][table.clamp(min=0).long()].reshape(n, -1, LATENT + ROPE).float()
    rows = q[index].float().reshape(n, most * heads, LATENT + ROPE)
    scores = torch.matmul(rows, keys.transpose(1, 2)).mul_(SCALE).reshape(n, most, heads, -1)
    j = torch.arange(keys.shape[1], device=q.device)
    seen = j <= ((seq - new)[:, None] + i)[:, :, None]
    seen &= j < seq[:, None, None]
    weights, norm, lse = _softmax(scores, seen[:, :, None])
    out = torch.matmul(weights.reshape(n, most * heads, -1), keys[..., :LATENT]).reshape(n, most, heads, LATENT)
    out = torch.where(norm > 0, out / norm, 0.0)
    return out[r, at].to(q.dtype), lse[r, at].contiguous()


def _plain_expanded(s):
    """softmax(scale (q_nope k_nope^T + q_rope k_rope^T)) v, request by request as the lengths say, a few heads at a time."""
    q, heads, n = s["q"], s["heads"], s["n"]
    cu_k = s["cu_seqlens_k"].long()
    new, count = (s["cu_seqlens"][1:] - s["cu_seqlens"][:-1]).long(), cu_k[1:] - cu_k[:-1]
    r, at, index, i = _rows_of(s)
    j = torch.arange(s["max_keys"], device=q.device)
    held = (cu_k[:-1, None] + j).clamp(max=max(0, s["v"].shape[0] - 1))
    seen = (j < count[:, None])[:, None]
    if s["causal"]:
        seen = seen & (j <= ((count - new)[:, None] + i)[:, :, None])
    outs, lses = [], []
    step = max(1, int(2e9 / max(1, n * s["max_new"] * s["max_keys"])))
    part = s["k_rope"][held].float()
    for h in range(0, heads, step):
        hs = slice(h, h + step)
        rows = q[:, hs][index].float().transpose(1, 2)                          # [n, heads, new, 192]
        k, v = s["k_nope"][:, hs][held].float().transpose(1, 2), s["v"][:, hs][held].float().transpose(1, 2)
        scores = torch.matmul(rows[..., :NOPE], k.transpose(2, 3))
        scores.add_(torch.matmul(rows[..., NOPE:], part[:, None].transpose(2, 3))).mul_(SCALE)
        weights, norm, lse = _softmax(scores, seen[:, None])
        out = torch.where(norm > 0, torch.matmul(weights, v) / norm, 0.0)
        outs.append(out.transpose(1, 2)[r, at])
        lses.append(lse.transpose(1, 2)[r, at])
    return torch.cat(outs, 1).to(q.dtype), torch.cat(lses, 1)


_plain = {"rotary": _plain_rotary, "append": _plain_append, "absorbed": _plain_absorbed, "expanded": _plain_expanded}


# ------------------------------------------------------------------ work
def work(case):
    """What one pass cannot do without: each input read once, each output written once, the products of visible keys."""
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rotary":
        n, heads = case["n"], case["heads"]
        return {"bytes": n * (2 * heads * case["dim"] * size + 4) + 2 * case["rot"], "flops": 3 * n * heads * case["rot"]}
    if case["op"] == "append":
        turn = 4 if case["rotated"] else 0
        return {"bytes": case["n"] * (2 * (LATENT + ROPE) * size + 8 + turn), "flops": 3 * case["n"] * ROPE if turn else 0}
    heads, bytes_, seen = case["heads"], 0, 0
    for ctx, new in _lengths(case):
        if case["op"] == "absorbed":
            bytes_ += (ctx + new if new else 0) * (LATENT + ROPE) * size + new * heads * ((2 * LATENT + ROPE) * size + 4)
        else:
            bytes_ += (ctx + new if new else 0) * (heads * (NOPE + VALUE) + ROPE) * size
            bytes_ += new * heads * ((NOPE + ROPE + VALUE) * size + 4)
        seen += new * ctx + (new * (new + 1) // 2 if case.get("causal", True) else new * new)
    per = 2 * (2 * LATENT + ROPE) if case["op"] == "absorbed" else 2 * (NOPE + ROPE + VALUE)
    return {"bytes": bytes_, "flops": per * seen * heads}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    if case["op"] in ("absorbed", "expanded") and work(case)["flops"] > 6e12:
        return None
    return _exact[case["op"]](prepare(case, seed))


def _exact_turned(x, positions, inv_freq, factor, interleaved):
    """Channel pairs as complex numbers, times factor * exp(i * position * frequency)."""
    half = inv_freq.numel()
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    z = torch.complex(x[..., first].double(), x[..., second].double())
    angle = torch.outer(positions.double(), inv_freq.double())
    z = z * torch.polar(torch.full_like(angle, factor), angle)[:, None, :]
    out = x.double().clone()
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_rotary(s):
    return _exact_turned(s["x"], s["positions"], s["inv_freq"], s["factor"], s["interleaved"])


def _exact_append(s):
    """The cache as flat rows."""
    flat, live = s["cache"].double().reshape(-1, LATENT + ROPE), torch.nonzero(s["slot_map"] >= 0)[:, 0]
    part = s["k_rope"].double()
    if s["rotated"]:
        part = _exact_turned(s["k_rope"][:, None], s["positions"], s["inv_freq"], 1.0, s["interleaved"])[:, 0]
    flat[s["slot_map"][live], :LATENT] = s["c"][live].double()
    flat[s["slot_map"][live], LATENT:] = part[live]
    return flat.reshape(s["cache"].shape)


def _exact_head(q, k, v, first, out, lse):
    """One head of one request: row i sees keys 0 ... first + i."""
    a = (q.double() @ k.double().T) * SCALE
    i, j = torch.arange(q.shape[0], device=q.device), torch.arange(k.shape[0], device=q.device)
    a.masked_fill_(j > first + i[:, None], -math.inf)
    lse.copy_(torch.logsumexp(a, dim=1))
    p = torch.exp(a - lse[:, None])
    out.copy_(torch.nan_to_num(p, nan=0.0) @ v.double())


def _exact_empty(s, width):
    q = s["q"]
    return (torch.zeros(*q.shape[:2], width, dtype=torch.float64, device=q.device),
            torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device))


def _exact_absorbed(s):
    out, lse = _exact_empty(s, LATENT)
    cu = s["cu_seqlens"].tolist()
    for n, end in enumerate(s["seq_len"].tolist()):
        a, b = cu[n], cu[n + 1]
        if a == b or end == 0:
            continue
        rows = s["cache"][s["block_table"][n, :_up(end, s["page"])].long()].reshape(-1, LATENT + ROPE)[:end]
        for h in range(s["heads"]):
            _exact_head(s["q"][a:b, h], rows, rows[:, :LATENT], end - (b - a), out[a:b, h], lse[a:b, h])
    return out, lse


def _exact_expanded(s):
    out, lse = _exact_empty(s, VALUE)
    cu, cu_k = s["cu_seqlens"].tolist(), s["cu_seqlens_k"].tolist()
    for n in range(s["n"]):
        a, b, x, y = cu[n], cu[n + 1], cu_k[n], cu_k[n + 1]
        if a == b or x == y:
            continue
        for h in range(s["heads"]):
            k = torch.cat([s["k_nope"][x:y, h], s["k_rope"][x:y]], dim=1)
            _exact_head(s["q"][a:b, h], k, s["v"][x:y, h], (y - x) - (b - a) if s["causal"] else y - x, out[a:b, h], lse[a:b, h])
    return out, lse


_exact = {"rotary": _exact_rotary, "append": _exact_append, "absorbed": _exact_absorbed, "expanded": _exact_expanded}
