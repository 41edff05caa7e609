"""Cases and plain forms of the serving-step operators that run beside the KDA layers.

A model that mixes KDA layers with softmax-attention layers serves its
requests in steps.  One step lays out the pages of every request
(``tables``), writes the new tokens' keys and values into the paged cache
(``append``), attends from the new tokens over that cache (``attention``) and,
when tokens were drafted, decides how many of them stand (``verify``) -- the
number that ``kda_decode_multi`` then commits to the recurrent state.

``listed()`` and ``draw()`` give cases, ``prepare()`` what a serving program
holds before a call, ``run()`` one pass through one operator: in plain torch
where ``own`` is false, through this package's entry points where it is true.
``exact()`` computes the same from the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a handful of decode requests, one token each: latency is all there is
        dict(name="tables_decode", op="tables", n=24, ctx_lo=5, ctx_hi=9000, new_lo=1, new_hi=1, page=16),
        # prompts of many lengths arriving together, a million tokens in all
        dict(name="tables_prompts", op="tables", n=320, ctx_lo=0, ctx_hi=30000, new_lo=33, new_hi=16384, page=64),
        # one decode step of a mid-sized batch
        dict(name="append_decode", op="append", n=96, heads=8, dim=128, page=16, dtype="bf16", pages=8192),
        # the keys and values of a long prompt chunk
        dict(name="append_prompt", op="append", n=40001, heads=8, dim=128, page=64, dtype="bf16", pages=2048),
        # a few short conversations, one token each
        dict(name="attn_decode_few", op="attention", n=4, ctx_lo=90, ctx_hi=1500, new_lo=1, new_hi=1, heads=32,
             kv_heads=8, dim=128, page=16, window=0, dtype="bf16"),
        # a full decode batch over long contexts: the cache is read once
        dict(name="attn_decode_batch", op="attention", n=64, ctx_lo=1024, ctx_hi=16384, new_lo=1, new_hi=1, heads=32,
             kv_heads=8, dim=128, page=64, window=0, dtype="bf16"),
        # the verify step of speculative decoding: eight tokens of each request
        dict(name="attn_verify", op="attention", n=32, ctx_lo=700, ctx_hi=8192, new_lo=8, new_hi=8, heads=32,
             kv_heads=4, dim=128, page=32, window=0, dtype="bf16"),
        # a long prompt taken in chunks, each chunk over all that came before
        dict(name="attn_chunk", op="attention", n=2, ctx_lo=12000, ctx_hi=27001, new_lo=4096, new_hi=4096, heads=32,
             kv_heads=4, dim=128, page=64, window=0, dtype="bf16"),
        # prompts and decode requests mixed, a sliding window, smaller heads
        dict(name="attn_window_mixed", op="attention", n=16, ctx_lo=0, ctx_hi=8000, new_lo=1, new_hi=513, heads=16,
             kv_heads=8, dim=64, page=32, window=1024, dtype="bf16"),
        # 32-bit numbers throughout, ragged
        dict(name="attn_fp32", op="attention", n=6, ctx_lo=17, ctx_hi=2100, new_lo=1, new_hi=65, heads=8, kv_heads=2,
             dim=64, page=16, window=0, dtype="fp32"),
        # a few requests over a small vocabulary
        dict(name="verify_few", op="verify", n=4, k=4, vocab=32000, dtype="fp32", one_hot=False),
        # a batch over a large vocabulary, seven drafted tokens each
        dict(name="verify_batch", op="verify", n=128, k=7, vocab=160001, dtype="fp32", one_hot=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "attention", "attention", "attention", "verify"])
    if op == "tables":
        n = _log(rng, 1, 320)
        new_hi = _log(rng, 1, 1000000 // n if n > 61 else 16384)
        return dict(op=op, n=n, ctx_lo=rng.choice([0, 1, 100]), ctx_hi=_log(rng, 101, 30000),
                    new_lo=rng.choice([0, 1]), new_hi=new_hi, page=rng.choice([16, 32, 64, 128]))
    if op == "append":
        n, page = _log(rng, 1, 40001), rng.choice([16, 32, 64, 128])
        return dict(op=op, n=n, heads=rng.choice([1, 2, 4, 8]), dim=rng.choice([32, 64, 128]), page=page,
                    dtype=rng.choice(["bf16", "bf16", "fp32"]), pages=_up(n, page) + rng.randint(8, 1024))
    if op == "verify":
        return dict(op=op, n=_log(rng, 1, 128), k=rng.randint(1, 7), vocab=_log(rng, 1000, 160001),
                    dtype=rng.choice(["fp32", "fp32", "bf16"]), one_hot=rng.random() < 0.25)
    kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8])
    shape = dict(heads=kv_heads * group, kv_heads=kv_heads, dim=rng.choice([32, 64, 128, 128]),
                 page=rng.choice([16, 32, 64, 128]), window=rng.choice([0, 0, _log(rng, 16, 4096)]),
                 dtype=rng.choice(["bf16", "bf16", "bf16", "fp32"]))
    kind = rng.choice(["decode", "verify", "chunk"])
    if kind == "decode":
        return dict(op=op, n=_log(rng, 1, 64), ctx_lo=rng.choice([0, 1, 300]), ctx_hi=_log(rng, 301, 16384), new_lo=1,
                    new_hi=1, **shape)
    if kind == "verify":
        new = rng.randint(2, 16)
        return dict(op=op, n=_log(rng, 1, 32), ctx_lo=rng.choice([0, 1, 300]), ctx_hi=_log(rng, 301, 8192),
                    new_lo=new, new_hi=new, **shape)
    wide = shape["dtype"] == "bf16"
    return dict(op=op, n=rng.randint(1, 4 if wide else 3), ctx_lo=0, ctx_hi=_log(rng, 64, 12000 if wide else 3000),
                new_lo=rng.choice([1, 17]), new_hi=_log(rng, 64, 2500 if wide else 700), **shape)


def _spread(lo, hi, n):
    """n lengths from lo to hi, spread over their logarithm."""
    if n == 1:
        return [hi]
    a, b = math.log(lo + 1), math.log(hi + 1)
    return [int(round(math.exp(a + (b - a) * i / (n - 1)))) - 1 for i in range(n)]


def _lengths(case):
    """(cached tokens, new tokens) of each request: the case's alone, in no particular order."""
    n = case["n"]
    ctx, new = _spread(case["ctx_lo"], case["ctx_hi"], n), _spread(case["new_lo"], case["new_hi"], n)
    step = next(s for s in range(n // 2 + 1, 2 * n + 2) if math.gcd(s, n) == 1)
    return [(ctx[i], new[(i * step) % n]) for i in range(n)]


def _up(a, b):
    return -(-a // b)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    state = dict(case)
    if case["op"] in ("tables", "attention"):
        _prepare_requests(state, gen)
    if case["op"] == "tables":
        return state
    if case["op"] == "append":
        dt, n, slots = DTYPES[case["dtype"]], case["n"], case["pages"] * case["page"]
        rows = lambda: torch.randn(n, case["heads"], case["dim"], generator=gen, device="cuda").to(dt)  # noqa: E731
        state["k"], state["v"] = rows(), rows()
        shape = (case["pages"], case["heads"], case["page"], case["dim"])
        state["k_cache"], state["v_cache"] = torch.zeros(shape, dtype=dt, device="cuda"), torch.zeros(shape, dtype=dt, device="cuda")
        state["slot_map"] = torch.randperm(slots, generator=gen, device="cuda")[:n].contiguous()
        if n > 8:
            state["slot_map"][-3:] = -1                 # padding of a fixed-size step
        return state
    if case["op"] == "attention":
        dt, total = DTYPES[case["dtype"]], int(state["total_new"])
        rows = lambda *shape: torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(dt)  # noqa: E731
        state["q"] = rows(total, case["heads"], case["dim"])
        shape = (state["n_pages"], case["kv_heads"], case["page"], case["dim"])
        state["k_cache"], state["v_cache"] = rows(*shape), rows(*shape)
        state["scale"] = case["dim"] ** -0.5
        return state
    # verify: the target's logits are the draft's with some noise, the drafted tokens are drawn from the draft
    n, k, vocab, dt = case["n"], case["k"], case["vocab"], DTYPES[case["dtype"]]
    logits = 2.0 * torch.randn(n, k, vocab, generator=gen, device="cuda")
    noise = torch.randn(n, k + 1, vocab, generator=gen, device="cuda")
    noise[:, :k].mul_(0.7).add_(logits)
    state["target"] = torch.softmax(noise, dim=-1).to(dt)
    del noise
    draft = torch.softmax(logits, dim=-1)
    if case["one_hot"]:
        state["tokens"] = torch.argmax(logits, dim=-1).to(torch.int32)
        state["draft"] = None
    else:
        at = torch.rand(n, k, 1, generator=gen, device="cuda", dtype=torch.float64)
        run_sum = torch.cumsum(draft.double(), dim=-1)
        state["tokens"] = torch.searchsorted(run_sum, at * run_sum[..., -1:]).clamp_(max=vocab - 1)[..., 0].to(torch.int32).contiguous()
        state["draft"] = draft.to(dt)
    state["uniforms"] = torch.rand(n, k + 1, generator=gen, device="cuda")
    state["draft_len"] = torch.randint(max(0, k - 2), k + 1, (n,), generator=gen, device="cuda", dtype=torch.int32)
    return state


def _prepare_requests(state, gen):
    """Lengths, pages and block tables of a step's requests, shuffled by the seed."""
    n, page = state["n"], state["page"]
    pairs = torch.tensor(_lengths(state), dtype=torch.int32, device="cuda")
    pairs = pairs[torch.randperm(n, generator=gen, device="cuda")]
    ctx, new = pairs[:, 0].contiguous(), pairs[:, 1].contiguous()
    lens = _lengths(state)
    total_new, used = sum(b for _, b in lens), sum(_up(a + b, page) for a, b in lens)
    blocks = max(1, max(_up(a + b, page) for a, b in lens))
    n_pages = used + 16
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    state.update(ctx_len=ctx, new_len=new, total_new=total_new, n_pages=n_pages, max_new=max(b for _, b in lens))
    col = torch.arange(blocks, device="cuda")[None, :]
    held = ctx if state["op"] == "tables" else ctx + new       # the pages that the requests hold already
    have = (held + page - 1) // page
    first = torch.cumsum(have, 0) - have
    table = torch.where(col < have[:, None], order[(first[:, None] + col).clamp(max=n_pages - 1)], -1)
    state["block_table"] = table.to(torch.int32).contiguous()
    state["free_pages"] = order[int(have.sum()):].contiguous()
    if state["op"] == "tables":                                # the fixed buffers of a serving step
        state["n_tokens"] = max(64, _up(total_new, 64) * 64)
        state["cu_seqlens"] = torch.empty(n + 1, dtype=torch.int32, device="cuda")
        state["seq_len"] = torch.empty(n, dtype=torch.int32, device="cuda")
        state["slot_map"] = torch.empty(state["n_tokens"], dtype=torch.int64, device="cuda")
        state["positions"] = torch.empty(state["n_tokens"], dtype=torch.int32, device="cuda")
        state["n_taken"] = torch.empty(1, dtype=torch.int32, device="cuda")
    else:
        state["cu_seqlens"] = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
        state["cu_seqlens"][1:] = torch.cumsum(new, 0)
        state["seq_len"] = (ctx + new).contiguous()


# ------------------------------------------------------------------ one pass
def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _own_tables(s):
    import kimi_delta_attention_chunked_gb300 as kda
    out = kda.kda_build_block_tables(s["ctx_len"], s["new_len"], s["free_pages"], s["block_table"], s["page"],
                                     s["n_tokens"], cu_seqlens=s["cu_seqlens"], seq_len=s["seq_len"],
                                     slot_map=s["slot_map"], positions=s["positions"], n_taken=s["n_taken"])
    return (s["block_table"], *out)


def _own_append(s):
    import kimi_delta_attention_chunked_gb300 as kda
    kda.kda_cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slot_map"])
    return s["k_cache"], s["v_cache"]


def _own_attention(s):
    import kimi_delta_attention_chunked_gb300 as kda
    return kda.kda_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["cu_seqlens"],
                                   s["seq_len"], scale=s["scale"], window=s["window"], want_lse=True)


def _own_verify(s):
    import kimi_delta_attention_chunked_gb300 as kda
    return kda.kda_verify_draft(s["target"], s["draft"], s["tokens"], s["uniforms"], s["draft_len"])


_own = {"tables": _own_tables, "append": _own_append, "attention": _own_attention, "verify": _own_verify}


def _plain_tables(s):
    """Pages are taken from the free list in request order; a token's slot is its page's start plus its place there."""
    page, table, free, n_tokens = s["page"], s["block_table"], s["free_pages"], s["n_tokens"]
    ctx, new = s["ctx_len"].long(), s["new_len"].long()
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=ctx.device), torch.cumsum(new, 0)])
    seq = ctx + new
    blocks = table.shape[1]
    have = ((ctx + page - 1) // page).clamp(max=blocks)
    need = ((seq + page - 1) // page).clamp(max=blocks) - have
    first = torch.cumsum(need, 0) - need
    col = torch.arange(blocks, device=ctx.device)[None, :]
    at = first[:, None] + col - have[:, None]
    fresh = torch.where(at < free.numel(), free[at.clamp(0, max(0, free.numel() - 1))], -1)
    table.copy_(torch.where((col >= have[:, None]) & (col < (have + need)[:, None]), fresh, table))
    t = torch.arange(n_tokens, device=ctx.device)
    live = t < cu[-1]
    r = torch.searchsorted(cu[1:], t, right=True).clamp(max=ctx.numel() - 1)
    pos = ctx[r] + t - cu[r]
    held = table[r, (pos // page).clamp(0, blocks - 1)].long()
    slot = torch.where(live & (held >= 0) & (pos < blocks * page), held * page + pos % page, -1)
    return (table, cu.to(torch.int32), seq.to(torch.int32), slot, torch.where(live, pos, 0).to(torch.int32),
            need.sum().reshape(1).to(torch.int32))


def _plain_append(s):
    """Row t of k and v goes to place slot % page of page slot // page; a negative slot is skipped."""
    k_cache, v_cache, page, slot = s["k_cache"], s["v_cache"], s["page"], s["slot_map"]
    live = slot >= 0
    slot = torch.where(live, slot, slot.amax())         # a skipped row writes what the last slot's own row writes
    row = torch.where(live, torch.arange(slot.numel(), device=slot.device), slot.argmax())
    k_cache[slot // page, :, slot % page] = s["k"][row]
    v_cache[slot // page, :, slot % page] = s["v"][row]
    return k_cache, v_cache


def _plain_attention(s):
    """softmax(scale q k^T) v of each new token over the keys up to its own position (the last `window` of them)."""
    q, table, cu, seq, page = s["q"], s["block_table"], s["cu_seqlens"].long(), s["seq_len"].long(), s["page"]
    n, kvh, dim = table.shape[0], s["kv_heads"], s["dim"]
    group, most, total = s["heads"] // kvh, s["max_new"], q.shape[0]
    held = table.clamp(min=0).long()
    keys = s["k_cache"][held].transpose(1, 2).reshape(n, kvh, -1, dim).float()
    values = s["v_cache"][held].transpose(1, 2).reshape(n, kvh, -1, dim).float()
    new = cu[1:] - cu[:-1]
    i = torch.arange(most, device=q.device)
    rows = q[(cu[:-1, None] + i).clamp(max=total - 1)].float()                      # [n, most, heads, dim]
    rows = rows.reshape(n, most, kvh, group, dim).permute(0, 2, 3, 1, 4).reshape(n, kvh, group * most, dim)
    scores = torch.matmul(rows, keys.transpose(2, 3)).mul_(s["scale"]).reshape(n, kvh, group, most, -1)
    pos = ((seq - new)[:, None] + i)[:, :, None]                                    # [n, most, 1]
    j = torch.arange(keys.shape[2], device=q.device)
    seen = (j <= pos) & (j < seq[:, None, None])
    if s["window"] > 0:
        seen &= j > pos - s["window"]
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    weights = scores.sub_(top).exp_()
    norm = weights.sum(dim=-1, keepdim=True)
    lse = (top + torch.log(norm))[..., 0]
    out = torch.matmul(weights.reshape(n, kvh, group * most, -1), values).reshape(n, kvh, group, most, dim)
    out = torch.where(norm > 0, out / norm, 0.0)
    t = torch.arange(total, device=q.device)
    r = torch.searchsorted(cu[1:], t, right=True)
    at = t - cu[r]
    o = out[r, :, :, at].reshape(total, s["heads"], dim)
    return o.to(q.dtype), lse[r, :, :, at].reshape(total, s["heads"])


def _plain_verify(s):
    """Draft i stands while u_i q_i < p_i; the next token is drawn from max(p - q, 0), or from p where all stand."""
    p, q, tokens, u = s["target"], s["draft"], s["tokens"].long(), s["uniforms"]
    n, k = tokens.shape
    vocab = p.shape[2]
    live = torch.arange(k, device=p.device) < s["draft_len"][:, None]
    pt = p[:, :k].gather(2, tokens[..., None])[..., 0].double()
    qt = torch.ones_like(pt) if q is None else q.gather(2, tokens[..., None])[..., 0].double()
    stands = live & (u[:, :k].double() * qt < pt)
    count = torch.cumprod(stands.long(), dim=1).sum(dim=1)
    request = torch.arange(n, device=p.device)
    row = p[request, count].double()
    at = count.clamp(max=k - 1)
    if q is None:
        off = torch.arange(vocab, device=p.device) == tokens[request, at][:, None]
        left = torch.where(off, (row - 1).clamp(min=0), row)
    else:
        left = (row - q[request, at].double()).clamp(min=0)
    left = torch.where((count < s["draft_len"])[:, None], left, row)
    left = torch.where(left.sum(dim=1, keepdim=True) > 0, left, row)
    run_sum = torch.cumsum(left, dim=1)
    drawn = (run_sum <= u[:, k:].double() * run_sum[:, -1:]).sum(dim=1)
    last = vocab - 1 - torch.argmax((left > 0).flip(1).to(torch.int8), dim=1)
    drawn = torch.minimum(drawn, last)
    i = torch.arange(k + 1, device=p.device)
    padded = torch.cat([tokens, tokens[:, :1]], dim=1)
    out = torch.where(i < count[:, None], padded, torch.where(i == count[:, None], drawn[:, None], -1))
    return out.to(torch.int32), (count + 1).to(torch.int32)


_plain = {"tables": _plain_tables, "append": _plain_append, "attention": _plain_attention, "verify": _plain_verify}


# ------------------------------------------------------------------ work
def work(case):
    """What one pass cannot do without: each input read once, each output written once, the products of visible keys."""
    if case["op"] == "tables":
        lens, page = _lengths(case), case["page"]
        taken = sum(_up(a + b, page) - _up(a, page) for a, b in lens)
        total = sum(b for _, b in lens)
        return {"bytes": 16 * case["n"] + 8 * taken + 12 * total, "flops": 0}
    if case["op"] == "append":
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": case["n"] * (4 * case["heads"] * case["dim"] * size + 8), "flops": 0}
    if case["op"] == "verify":
        size = 2 if case["dtype"] == "bf16" else 4
        rows = 1 if case["one_hot"] else 2
        return {"bytes": case["n"] * (rows * case["vocab"] * size + 16 * (case["k"] + 1)), "flops": 2 * case["n"] * case["vocab"]}
    size, window = 2 if case["dtype"] == "bf16" else 4, case["window"]
    bytes_, seen = 0, 0
    for ctx, new in _lengths(case):
        first = max(0, ctx + 1 - window) if window else 0
        bytes_ += 2 * (ctx + new - first if new else 0) * case["kv_heads"] * case["dim"] * size
        bytes_ += new * case["heads"] * (2 * case["dim"] * size + 4)
        full = max(0, min(new, window - ctx)) if window else new        # tokens that the window does not cut
        seen += full * ctx + full * (full + 1) // 2 + (new - full) * window
    return {"bytes": bytes_, "flops": 4 * seen * case["heads"] * case["dim"]}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    return _exact[case["op"]](prepare(case, seed))


def _exact_tables(s):
    """Request by request, token by token, on the host."""
    ctx, new, free, page = s["ctx_len"].tolist(), s["new_len"].tolist(), s["free_pages"].tolist(), s["page"]
    table, blocks = s["block_table"].tolist(), s["block_table"].shape[1]
    cu, seq, slots, places, taken = [0], [], [], [], 0
    for n in range(len(ctx)):
        end = ctx[n] + new[n]
        for b in range(_up(ctx[n], page), min(_up(end, page), blocks)):
            table[n][b] = free[taken] if taken < len(free) else -1
            taken += 1
        for pos in range(ctx[n], end):
            b = pos // page
            slots.append(table[n][b] * page + pos % page if b < blocks and table[n][b] >= 0 else -1)
            places.append(pos)
        cu.append(cu[-1] + new[n])
        seq.append(end)
    pad = s["n_tokens"] - len(slots)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return (i32(table), i32(cu), i32(seq), torch.tensor(slots + [-1] * pad, dtype=torch.int64), i32(places + [0] * pad), i32([taken]))


def _exact_append(s):
    """The caches as flat rows: a live row's place is its page's start, its head's, then its own."""
    slot, page, heads, dim = s["slot_map"], s["page"], s["heads"], s["dim"]
    live = torch.nonzero(slot >= 0)[:, 0]
    base = (slot[live] // page) * heads * page + slot[live] % page
    at = (base[:, None] + torch.arange(heads, device=slot.device) * page).reshape(-1)
    out = []
    for rows, cache in ((s["k"], s["k_cache"]), (s["v"], s["v_cache"])):
        flat = cache.reshape(-1, dim).clone()
        flat.index_copy_(0, at, rows[live].reshape(-1, dim))
        out.append(flat.reshape(cache.shape))
    return tuple(out)


def _exact_attention(s):
    """Request by request and head by head, in 64 bits, over the keys in their order."""
    q, page, window, cu = s["q"], s["page"], s["window"], s["cu_seqlens"].tolist()
    heads, kvh, dim = s["heads"], s["kv_heads"], s["dim"]
    lens = _lengths(case=s)
    if 4 * heads * dim * sum(b * (a + b) for a, b in lens) > 8e12:
        return None
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full((q.shape[0], heads), -math.inf, dtype=torch.float64, device=q.device)
    for n, end in enumerate(s["seq_len"].tolist()):
        m = cu[n + 1] - cu[n]
        if m == 0 or end == 0:
            continue
        held = s["block_table"][n, :_up(end, page)].long()
        at, j = torch.arange(end - m, end, device=q.device)[:, None], torch.arange(end, device=q.device)[None]
        hidden = (j > at) | (j <= at - window) if window else j > at
        for h in range(kvh):
            k = s["k_cache"][held, h].reshape(-1, dim)[:end].double()
            v = s["v_cache"][held, h].reshape(-1, dim)[:end].double()
            for g in range(h * (heads // kvh), (h + 1) * (heads // kvh)):
                a = (q[cu[n]:cu[n + 1], g].double() @ k.T) * s["scale"]
                a[hidden] = -math.inf
                lse[cu[n]:cu[n + 1], g] = torch.logsumexp(a, dim=1)
                out[cu[n]:cu[n + 1], g] = torch.exp(a - lse[cu[n]:cu[n + 1], g, None]) @ v
    return out, lse


def _exact_verify(s):
    """Request by request; the drawn token by bisection in the running sum."""
    p, q, tokens, u = s["target"], s["draft"], s["tokens"].tolist(), s["uniforms"].double().cpu()
    k, vocab = s["k"], p.shape[2]
    out, commit = [], []
    for n, length in enumerate(s["draft_len"].tolist()):
        a = 0
        while a < length:
            pa = float(p[n, a, tokens[n][a]])
            qa = 1.0 if q is None else float(q[n, a, tokens[n][a]])
            if not float(u[n, a]) * qa < pa:
                break
            a += 1
        row = p[n, a].double()
        left = row.clone()
        if a < length:
            if q is None:
                left[tokens[n][a]] = max(0.0, float(row[tokens[n][a]]) - 1.0)
            else:
                left = torch.relu(row - q[n, a].double())
            if not float(left.sum()) > 0:
                left = row
        run_sum = torch.cumsum(left, 0)
        x = int(torch.searchsorted(run_sum, run_sum[-1:] * u[n, k].to(p.device), right=True))
        x = min(x, int(torch.nonzero(left > 0)[-1]))
        out.append(tokens[n][:a] + [x] + [-1] * (k - a))
        commit.append(a + 1)
    return torch.tensor(out, dtype=torch.int32), torch.tensor(commit, dtype=torch.int32)


_exact = {"tables": _exact_tables, "append": _exact_append, "attention": _exact_attention, "verify": _exact_verify}
