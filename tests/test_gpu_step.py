"""The serving-step operators on the GPU against their 64-bit plain forms
(tests/_step.py): block tables, cache append, paged attention, verification."""
import math

import pytest
import torch

from _gpu import need_gpu
from _step import HALF, attention_ref, lay_out, tables_ref, verify_ref

import kimi_delta_attention_chunked_gb300 as kda

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


# ------------------------------------------------------------------ tables
@pytest.mark.parametrize("ctx,new,page,n_free,blocks,pad", [
    ([0], [1], 16, 4, 4, 0),
    ([15, 16, 17], [1, 1, 1], 16, 8, 4, 61),
    ([0, 0, 0, 0], [0, 0, 0, 0], 32, 3, 2, 5),
    ([5, 0, 64, 3], [0, 130, 1, 0], 64, 9, 4, 1),
    ([100, 7], [50, 300], 16, 5, 32, 3),                    # the free list runs out
    ([10, 40], [30, 90], 16, 30, 5, 0),                     # tokens past the table
    ([-4, 3], [6, -2], 16, 9, 3, 2),                        # negative lengths count as 0
    ([31] * 700, [1, 2, 33] * 233 + [5], 128, 1500, 3, 11),  # more requests than a block has threads
    (list(range(3000)), [0, 1] * 1500, 256, 1500, 20, 0),
], ids=lambda v: str(v)[:24])
def test_tables(ctx, new, page, n_free, blocks, pad):
    dev = need_gpu()
    gen = torch.Generator().manual_seed(1)
    n_tokens = sum(max(0, x) for x in new) + pad
    pool = torch.randperm(n_free + len(ctx) * blocks, generator=gen).tolist()
    free = pool[:n_free]
    table = [[pool[n_free + n * blocks + b] if b * page < ctx[n] else -1 for b in range(blocks)] for n in range(len(ctx))]
    t = i32(table, dev)
    cu, seq, slot, pos, taken = kda.kda_build_block_tables(i32(ctx, dev), i32(new, dev), i32(free, dev), t, page, n_tokens)
    r = tables_ref(ctx, new, free, table, page, n_tokens)
    assert t.tolist() == r[0] and cu.tolist() == r[1] and seq.tolist() == r[2]
    assert slot.tolist() == r[3] and pos.tolist() == r[4] and taken.tolist() == [r[5]]


def test_tables_short_slot_map_and_odd_buffers():
    """Fewer rows than new tokens, and buffers that are not 16-byte aligned."""
    dev = need_gpu()
    ctx, new, page = [3, 20, 0], [9, 14, 21], 16
    free = list(range(50, 60))
    table = [[1, -1], [2, 3], [-1, -1]]
    for n_tokens in (0, 1, 17, 43):
        t = i32(table, dev)
        slot = torch.empty(n_tokens + 1, dtype=torch.int64, device=dev)[1:]
        pos = torch.empty(n_tokens + 3, dtype=torch.int32, device=dev)[3:]
        cu, seq, slot, pos, taken = kda.kda_build_block_tables(i32(ctx, dev), i32(new, dev), i32(free, dev), t, page,
                                                               n_tokens, slot_map=slot, positions=pos)
        r = tables_ref(ctx, new, free, table, page, n_tokens)
        assert (t.tolist(), slot.tolist(), pos.tolist(), taken.tolist()) == (r[0], r[3], r[4], [r[5]])


def test_tables_no_requests():
    dev = need_gpu()
    e = torch.empty(0, dtype=torch.int32, device=dev)
    cu, seq, slot, pos, taken = kda.kda_build_block_tables(e, e, e, e.reshape(0, 4), 16, 6)
    assert cu.tolist() == [0] and slot.tolist() == [-1] * 6 and pos.tolist() == [0] * 6 and taken.tolist() == [0]


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,H,d,page,extra,skew", [
    (1, 1, 32, 16, 0, 0), (7, 2, 64, 16, 0, 0), (300, 8, 128, 64, 64, 0), (33, 3, 128, 32, 5, 0), (50, 2, 32, 256, 0, 1),
])
def test_append(dtype, T, H, d, page, extra, skew):
    """Contiguous rows, slices of wider rows (`extra` elements between tokens) and rows off
    a 16-byte boundary (`skew`); every other place of the cache stays as it was."""
    dev = need_gpu()
    gen = torch.Generator(device=dev).manual_seed(T + d)
    pages = -(-T // page) + 3
    wide = torch.randn(2, T, H * d + extra + skew, generator=gen, device=dev).to(dtype)
    k, v = (wide[x, :, skew:skew + H * d].unflatten(1, (H, d)) for x in (0, 1))
    kc, vc = (torch.randn(pages, H, page, d, generator=gen, device=dev).to(dtype) for _ in range(2))
    slot = torch.randperm(pages * page, generator=gen, device=dev)[:T].contiguous()
    if T > 5:
        slot[2], slot[3], slot[5] = -1, pages * page, -(1 << 40)
    ke, ve = kc.clone(), vc.clone()
    for t, s in enumerate(slot.tolist()):
        if 0 <= s < pages * page:
            ke[s // page, :, s % page] = k[t]
            ve[s // page, :, s % page] = v[t]
    kda.kda_cache_append(k, v, kc, vc, slot)
    assert torch.equal(kc, ke) and torch.equal(vc, ve)


def test_append_far_offsets():
    """Slots whose element offset passes 32 bits."""
    dev = need_gpu()
    H, page, d = 8, 256, 128
    pages = (1 << 32) // (H * page * d) + 40
    kc = torch.zeros(pages, H, page, d, dtype=BF, device=dev)
    vc = torch.zeros(pages, H, page, d, dtype=BF, device=dev)
    k, v = (torch.randn(3, H, d, device=dev).to(BF) for _ in range(2))
    slot = torch.tensor([pages * page - 1, 5, (pages // 2) * page + 9], device=dev)
    kda.kda_cache_append(k, v, kc, vc, slot)
    for t, s in enumerate(slot.tolist()):
        assert torch.equal(kc[s // page, :, s % page], k[t]) and torch.equal(vc[s // page, :, s % page], v[t])
    assert int(torch.count_nonzero(kc[:, 0, :, 0])) <= 3


# ------------------------------------------------------------------ attention
def make(lens, Hq, Hkv, d, page, dtype, dev, seed=0, blocks=None, n_extra=3, qpad=0):
    gen = torch.Generator().manual_seed(seed)
    table, cu, seq, n_pages = lay_out(lens, page, n_extra, gen, blocks)
    T = int(cu[-1])
    rnd = lambda *s: torch.randn(*s, generator=gen).to(dtype)  # noqa: E731
    wide = rnd(T, Hq * d + qpad)
    q = wide[:, qpad:].unflatten(1, (Hq, d))
    return dict(q=q, k=rnd(n_pages, Hkv, page, d), v=rnd(n_pages, Hkv, page, d), table=table, cu=cu, seq=seq,
                wide=wide, qpad=qpad)


def on(c, dev):
    wide = c["wide"].to(dev)
    q = wide[:, c["qpad"]:].unflatten(1, tuple(c["q"].shape[1:]))
    return [q] + [c[x].to(dev) for x in ("k", "v", "table", "cu", "seq")]


def check(c, dev, window=0, scale=None, **kw):
    """Runs the kernel and holds it to the bounds; returns (o, lse) on the CPU."""
    q = c["q"]
    s = q.shape[2] ** -0.5 if scale is None else scale
    o, lse = kda.kda_paged_attention(*on(c, dev), scale=s, window=window, want_lse=True, **kw)
    assert kda.kda_get_last_device_status() == 0
    ref, rl, bo, bl = attention_ref(q, c["k"], c["v"], c["table"], c["cu"], c["seq"], s, window)
    o, lse = o.double().cpu(), lse.double().cpu()
    rows = slice(0, int(c["cu"][-1]))
    bad = ~((o - ref).abs() <= bo)[rows]
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} outputs; worst {float(((o - ref).abs() - bo)[rows].max()):.2e}"
                           f" over its bound, first at {bad.nonzero()[0].tolist()}")
    empty = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse[rows]), empty[rows]) and bool((lse[empty] == -math.inf).all())
    assert bool(((lse - rl).abs() <= bl)[~empty].all())
    return o, lse


HEADS = [(1, 1), (4, 4), (8, 2), (8, 1), (6, 2), (32, 4)]


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (BF, 32), (F32, 32), (F32, 64), (F32, 128)])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_attention_mixed_lengths(dtype, d, Hq, Hkv):
    """Decode, verify and chunk rows in one call, with idle requests between them."""
    dev = need_gpu()
    lens = [(0, 1), (200, 1), (0, 0), (127, 1), (128, 1), (5, 0), (60, 7), (0, 70), (33, 40), (511, 2)]
    check(make(lens, Hq, Hkv, d, 16, dtype, dev, seed=d + Hq), dev)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64)])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_attention_pages(dtype, d, page):
    """Every page size; lengths on, below and above page and tile borders."""
    dev = need_gpu()
    lens = [(page - 1, 1), (page, 1), (2 * page - 2, 3), (127, 2), (255, 1), (256, 1), (300, 17), (0, page + 1)]
    check(make(lens, 4, 2, d, page, dtype, dev, seed=page), dev)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 128)])
@pytest.mark.parametrize("window", [1, 2, 16, 100, 128, 129, 1000])
def test_attention_window(dtype, d, window):
    dev = need_gpu()
    lens = [(0, 1), (700, 1), (300, 5), (0, 90), (250, 33), (17, 1)]
    check(make(lens, 8, 2, d, 32, dtype, dev, seed=window), dev, window=window)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (BF, 32), (F32, 64)])
def test_attention_long_chunks(dtype, d):
    """Chunks of several units per head over a context of several tiles; few heads of many
    rows, and many heads that share one."""
    dev = need_gpu()
    for Hq, Hkv, lens in ((2, 2, [(130, 300), (0, 270)]), (16, 1, [(500, 40), (1, 100)]), (3, 1, [(64, 129)])):
        check(make(lens, Hq, Hkv, d, 64, dtype, dev, seed=Hq), dev)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64)])
def test_attention_one_long_request(dtype, d):
    """One token over a long context: the context is split over the grid and joined."""
    dev = need_gpu()
    check(make([(9000, 1)], 8, 2, d, 64, dtype, dev, seed=3), dev)
    check(make([(4999, 3)], 4, 4, d, 16, dtype, dev, seed=4), dev)


@pytest.mark.parametrize("dtype,d,Hq,Hkv", [(BF, 64, 128, 1), (BF, 128, 66, 2), (F32, 32, 48, 1), (BF, 128, 200, 1),
                                             (BF, 64, 37, 1), (F32, 32, 37, 1)])
def test_attention_many_heads_share_one(dtype, d, Hq, Hkv):
    dev = need_gpu()
    check(make([(70, 3), (0, 5), (300, 1)], Hq, Hkv, d, 16, dtype, dev, seed=Hq), dev)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 32)])
def test_attention_rows_without_keys(dtype, d):
    """More new tokens than the sequence holds: the rows before position 0 see nothing."""
    dev = need_gpu()
    c = make([(-3, 5), (40, 2), (-200, 201), (-7, 7)], 4, 2, d, 16, dtype, dev)
    o, lse = check(c, dev)
    assert bool((o[:3] == 0).all()) and bool((lse[:3] == -math.inf).all())
    assert bool((o[-7:] == 0).all())
    # no table columns, no pages at all
    c = make([(0, 3)], 4, 2, d, 16, dtype, dev)
    c["table"] = c["table"][:, :0].contiguous()
    o, lse = check(c, dev)
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (BF, 32), (F32, 64)])
@pytest.mark.parametrize("page", [16, 128])
def test_attention_missing_pages(dtype, d, page):
    """Entries that name no page are left out, as are keys past the table."""
    dev = need_gpu()
    c = make([(400, 3), (400, 1), (600, 90), (150, 2)], 8, 2, d, page, dtype, dev)
    c["table"][0, 1] = -1
    c["table"][1, :] = -5
    c["table"][2, 2] = c["k"].shape[0]
    c["table"][2, 3] = 2 ** 31 - 1
    c["table"][3, 0] = -2 ** 31
    o, _ = check(c, dev)
    assert bool((o[3] == 0).all())
    c["table"] = c["table"][:, :3].contiguous()
    check(c, dev)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (BF, 32), (F32, 64)])
@pytest.mark.parametrize("window", [0, 50])
def test_attention_unseen_places_do_not_matter(dtype, d, window, bad):
    """NaN and infinities behind the last token, in pages of nobody, before the window and
    in tokens that come later leave every row that does not see them as it was."""
    dev = need_gpu()
    lens = [(37, 1), (250, 9), (0, 140), (129, 40)]
    c = make(lens, 8, 2, d, 32, dtype, dev, seed=9)
    clean = kda.kda_paged_attention(*on(c, dev), window=window, want_lse=True)
    page = 32
    used = torch.zeros(c["k"].shape[0], page, dtype=torch.bool)
    for n, (a, b) in enumerate(lens):
        for p in range(max(0, a - window + 1) if window else 0, a + b):
            used[int(c["table"][n, p // page]), p % page] = True
    for x in ("k", "v"):
        c[x].permute(0, 2, 1, 3)[~used] = bad
    got = kda.kda_paged_attention(*on(c, dev), window=window, want_lse=True)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])
    # the last token of each chunk holds it: only the rows at it see it
    for n, (a, b) in enumerate(lens):
        p = a + b - 1
        c["v"][int(c["table"][n, p // page]), :, p % page] = bad
    got = kda.kda_paged_attention(*on(c, dev), window=window, want_lse=True)
    last = (c["cu"][1:] - 1).tolist()
    others = [t for t in range(int(c["cu"][-1])) if t not in last]
    torch.testing.assert_close(got[0][others], clean[0][others], rtol=0, atol=0)
    assert not torch.isfinite(got[0][last]).any()
    if math.isnan(bad):
        assert torch.isnan(got[0][last]).all()
    else:
        assert bool((got[0][last] == bad).all())
    for n, (a, b) in enumerate(lens):
        p = a + b - 1
        c["k"][int(c["table"][n, p // page]), :, p % page] = math.nan
    got = kda.kda_paged_attention(*on(c, dev), window=window, want_lse=True)
    torch.testing.assert_close(got[0][others], clean[0][others], rtol=0, atol=0)
    assert torch.isnan(got[0][last]).all() and torch.isnan(got[1][last]).all()


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64)])
def test_attention_large_scores(dtype, d):
    """Scores far apart (a reference that moves by hundreds of octaves) and all equal."""
    dev = need_gpu()
    c = make([(500, 3), (0, 200)], 4, 2, d, 16, dtype, dev, seed=5)
    check(c, dev, scale=3.0)
    c["k"] *= torch.linspace(0.01, 8, c["k"].shape[0])[:, None, None, None].to(dtype)
    check(c, dev, scale=1.0)
    c["k"].zero_()
    check(c, dev)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64), (BF, 32)])
@pytest.mark.parametrize("qpad", [0, 8, 64, 3])
def test_attention_strided_q(dtype, d, qpad):
    """q as a slice of wider rows, on and off 16-byte boundaries; padding rows at the end are not written."""
    dev = need_gpu()
    c = make([(100, 2), (3, 9)], 4, 2, d, 16, dtype, dev, qpad=qpad)
    check(c, dev)
    args = on(c, dev)
    wide = c["wide"].to(dev)                               # the same strides and alignment, with rows behind the last token
    q = torch.cat([wide, torch.full_like(wide[:5], math.nan)])[:, qpad:].unflatten(1, (4, d))
    o = torch.full(tuple(q.shape), 7.0, dtype=dtype, device=dev)
    kda.kda_paged_attention(q, *args[1:], o=o)
    assert bool((o[-5:] == 7).all())
    assert torch.equal(o[:-5], kda.kda_paged_attention(*args))


def test_binding_refuses_layouts_the_kernels_cannot_read():
    """What only shows past the device check: strides, devices and dtypes."""
    dev = need_gpu()
    c = make([(20, 3)], 4, 2, 32, 16, F32, dev)
    args = on(c, dev)
    wide = torch.zeros(3, 8, 32, device=dev)
    for q in (wide[:, ::2], torch.zeros(3, 32, 4, device=dev).transpose(1, 2)):
        with pytest.raises(ValueError, match="contiguous"):
            kda.kda_paged_attention(q, *args[1:])
    with pytest.raises(ValueError, match="overlap"):
        kda.kda_paged_attention(torch.zeros(1, 4, 32, device=dev).expand(3, 4, 32), *args[1:])
    for i, word in ((1, "one shape|contiguous|k_cache"), (3, "block_table"), (4, "cu_seqlens"), (5, "seq_len")):
        bad = list(args)
        bad[i] = bad[i].cpu()
        with pytest.raises(ValueError, match=word):
            kda.kda_paged_attention(*bad)
    bad = list(args)
    bad[3] = bad[3].long()
    with pytest.raises(TypeError, match="block_table must be torch.int32, got torch.int64"):
        kda.kda_paged_attention(*bad)
    bad = list(args)
    bad[1] = bad[1].transpose(1, 2).contiguous().transpose(1, 2)
    with pytest.raises(ValueError, match="k_cache must be contiguous"):
        kda.kda_paged_attention(*bad)
    with pytest.raises(kda.KDAError, match="KDA_ERR_WORKSPACE"):
        kda.kda_paged_attention(*args, workspace=torch.empty(16, dtype=torch.uint8, device=dev))
    with pytest.raises(kda.KDAError, match="KDA_ERR_INVALID_ARG"):
        kda.kda_paged_attention(*args, scale=-1.0)
    slot = torch.zeros(3, dtype=torch.int64, device=dev)
    kv = torch.zeros(3, 4, 32, device=dev)
    with pytest.raises(ValueError, match="v: the heads of a token must be contiguous"):
        kda.kda_cache_append(kv[:, :2], kv[:, ::2], args[1], args[2], slot)
    with pytest.raises(TypeError, match="slot_map must be torch.int64"):
        kda.kda_cache_append(kv[:, :2], kv[:, :2], args[1], args[2], slot.int())
    with pytest.raises(TypeError, match="draft_len must be torch.int32"):
        p = torch.zeros(2, 2, 10, device=dev)
        kda.kda_verify_draft(p, None, torch.zeros(2, 1, dtype=torch.int32, device=dev), torch.zeros(2, 2, device=dev),
                             torch.zeros(2, device=dev))
    with pytest.raises(TypeError, match="must be a tensor"):
        kda.kda_verify_draft(None, None, None, None)


def test_attention_far_offsets():
    """A page whose element offset passes 32 bits, on both paths."""
    dev = need_gpu()
    for dtype, d, page, Hkv in ((BF, 128, 256, 8), (F32, 32, 256, 8)):
        n_pages = (1 << 32) // (Hkv * page * d) + 3
        kc = torch.zeros(n_pages, Hkv, page, d, dtype=dtype, device=dev)
        vc = torch.zeros(n_pages, Hkv, page, d, dtype=dtype, device=dev)
        c = make([(700, 2)], 16, Hkv, d, page, dtype, dev)
        small = on(c, dev)
        table = torch.tensor([[n_pages - 1, n_pages - 3, n_pages - 2]], dtype=torch.int32, device=dev)
        for b in range(3):
            kc[table[0, b]] = small[1][c["table"][0, b]]
            vc[table[0, b]] = small[2][c["table"][0, b]]
        got = kda.kda_paged_attention(small[0], kc, vc, table, small[4], small[5])
        assert torch.equal(got, kda.kda_paged_attention(*small))
        del kc, vc


def test_attention_device_lengths_out_of_range():
    """Offsets and lengths that leave the buffers are brought back into them."""
    dev = need_gpu()
    for dtype, d in ((BF, 128), (F32, 32)):
        c = make([(50, 4), (20, 6)], 4, 2, d, 16, dtype, dev)
        args = on(c, dev)
        args[4] = i32([-5, 4, 2 ** 31 - 1], dev)
        args[5] = i32([54, 26], dev)
        assert torch.equal(kda.kda_paged_attention(*args), kda.kda_paged_attention(*on(c, dev)))
        args[5] = i32([2 ** 31 - 1, -9], dev)
        o = kda.kda_paged_attention(*args)
        assert bool((o[4:] == 0).all())
        assert kda.kda_get_last_device_status() == 0


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_attention_other_stream_and_graph(dtype, d):
    """The same bits on another stream and from a captured graph whose lengths change."""
    dev = need_gpu()
    c = make([(300, 2), (90, 30), (5, 1)], 8, 2, d, 32, dtype, dev)
    args = on(c, dev)
    want = kda.kda_paged_attention(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = torch.empty_like(want)
    got = kda.kda_paged_attention(*args, o=o, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    ws = torch.empty(kda.kda_paged_attention_workspace_size(*args[0].shape[:2], 2, d, dtype), dtype=torch.uint8, device=dev)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        kda.kda_paged_attention(*args, o=o, workspace=ws)
    o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want)
    args[5].copy_(i32([150, 40, 6], dev))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, kda.kda_paged_attention(*args))


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_attention_memory_made_for_another_stream(dtype, d):
    """The workspace that a call on another stream makes is not handed out again before
    that stream has used it."""
    dev = need_gpu()
    c = make([(3000, 2), (2000, 30)], 8, 2, d, 32, dtype, dev)
    args = on(c, dev)
    want = kda.kda_paged_attention(*args)
    size = kda.kda_paged_attention_workspace_size(*args[0].shape[:2], 2, d, dtype)
    side = torch.cuda.Stream()
    o = torch.empty_like(want)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)                       # ~10 ms before the call's kernels
    kda.kda_paged_attention(*args, o=o, stream=side)
    junk = [torch.full((size,), 255, dtype=torch.uint8, device=dev) for _ in range(3)]
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and len(junk) == 3
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = kda.kda_verify_draft(torch.full((4, 2, 9), 1 / 9, device=dev), None, torch.zeros(4, 1, dtype=torch.int32, device=dev),
                               torch.zeros(4, 2, device=dev), stream=side)
    side.synchronize()
    assert got[1].tolist() == [2] * 4


def test_attention_many_requests():
    """As many requests as a step may have, most of them idle."""
    dev = need_gpu()
    lens = [(n % 40, 1 if n % 9 == 0 else 0) for n in range(8192)]
    for dtype, d in ((BF, 64), (F32, 32)):
        check(make(lens, 2, 1, d, 16, dtype, dev), dev)


# ------------------------------------------------------------------ verification
def dists(n, k, V, dtype, seed, sharp=2.0):
    gen = torch.Generator().manual_seed(seed)
    logits = sharp * torch.randn(n, k, V, generator=gen)
    draft = torch.softmax(logits, -1)
    t = torch.randn(n, k + 1, V, generator=gen)
    t[:, :k] = logits + 0.7 * t[:, :k]
    target = torch.softmax(t, -1)
    tokens = torch.multinomial(draft.reshape(n * k, V), 1, generator=gen).reshape(n, k).to(torch.int32) if k else torch.zeros(n, 0, dtype=torch.int32)
    return target.to(dtype), draft.to(dtype), tokens, torch.rand(n, k + 1, generator=gen)


def run_verify(target, draft, tokens, u, lens, dev):
    got = kda.kda_verify_draft(target.to(dev), None if draft is None else draft.to(dev), tokens.to(dev), u.to(dev),
                               None if lens is None else i32(lens, dev))
    k = tokens.shape[1]
    want = verify_ref(target, draft, tokens, u, [k] * target.shape[0] if lens is None else [min(max(x, 0), k) for x in lens])
    assert got[1].tolist() == want[1]
    assert got[0].tolist() == want[0]
    return got


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n,k,V", [(1, 1, 1), (3, 2, 7), (5, 4, 100), (4, 16, 1000), (2, 3, 33001), (40, 7, 513), (2, 0, 50)])
@pytest.mark.parametrize("one_hot", [False, True])
def test_verify(dtype, n, k, V, one_hot):
    dev = need_gpu()
    target, draft, tokens, u = dists(n, k, V, dtype, n + k + V)
    lens = [(i * 5) % (k + 1) for i in range(n)]
    run_verify(target, None if one_hot else draft, tokens, u, None, dev)
    run_verify(target, None if one_hot else draft, tokens, u, lens, dev)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_verify_edges(dtype):
    """Uniforms at 0 and next to 1, equal rows, zero rows, NaN, lengths and tokens out of range."""
    dev = need_gpu()
    for u_val in (0.0, 1.0 - 2.0 ** -24, 1.0):
        target, draft, tokens, u = dists(6, 3, 77, dtype, 3)
        u[:, -1] = u_val
        run_verify(target, draft, tokens, u, [-3, 0, 1, 2, 3, 9], dev)
    u.fill_(1.0)                                             # u q < p fails where p = q
    run_verify(draft_as_target(draft), draft, tokens, u, None, dev)
    target[2] = 0
    target[3, :, 10:] = math.nan
    draft[4, :, ::2] = math.nan
    target[5, :, 0] = -1.0
    tokens[0, 1], tokens[1, 0] = -1, 77
    u = torch.rand(6, 4, generator=torch.Generator().manual_seed(8))
    run_verify(target, draft, tokens, u, None, dev)
    run_verify(target, None, tokens, u, None, dev)


def draft_as_target(draft):
    return torch.cat([draft, draft[:, :1]], 1).contiguous()


def test_verify_tiny_probabilities():
    """A remainder of probabilities far below the kept ones is still drawn from exactly."""
    dev = need_gpu()
    V = 5000
    draft = torch.full((4, 1, V), 2.0 ** -34)
    draft[:, 0, 17] = 0.75
    target = torch.full((4, 2, V), 2.0 ** -33)
    target[:, 0, 17] = 0.25
    tokens = torch.full((4, 1), 17, dtype=torch.int32)
    u = torch.tensor([[0.9, 0.1], [0.9, 0.5], [0.9, 0.999], [0.2, 0.5]])
    got = run_verify(target, draft, tokens, u, None, dev)
    assert got[1].tolist() == [1, 1, 1, 2]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("V", [10, 700, 20002])
@pytest.mark.parametrize("with_draft", [False, True])
def test_verify_threshold_on_a_border(dtype, V, with_draft):
    """The running sum meets u times the whole sum exactly, or misses it by 2^-60: the
    sums of a row's halves are equal, but for one small element of one of them."""
    dev = need_gpu()
    gen = torch.Generator().manual_seed(V)
    half = V // 2
    target = torch.zeros(6, 1 + with_draft, V, dtype=dtype)
    for i in range(6):
        h = ((torch.rand(half, generator=gen) + 0.01) / V).to(dtype)
        h[half // 3] = 2.0 ** -53
        row = torch.cat([h, h[torch.randperm(half, generator=gen)]])
        more = 2.0 ** -53 * (1 + 2.0 ** -7) if not with_draft else 2.0 ** -52 * (1 + 2.0 ** -7)
        if with_draft:
            row[row == 2.0 ** -53] = 2.0 ** -52
        small = (row == (2.0 ** -52 if with_draft else 2.0 ** -53)).nonzero()[:, 0]
        assert small.numel() == 2
        if i % 3:
            row[small[i % 3 - 1]] = more
        target[i, 0] = row
    u = torch.full((6, 1 + with_draft), 0.5)
    tokens = torch.full((6, int(with_draft)), -1, dtype=torch.int32)
    got = run_verify(target, target[:, :1] / 2 if with_draft else None, tokens, u, None, dev)
    assert got[0][:, 0].tolist() == [half, half - 1, half] * 2
    u[:, -1] = 2.0 ** -140
    run_verify(target, None, tokens, u, None, dev)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_verify_threshold_is_not_rounded(dtype):
    """3/4 of the whole sum lies 20 x 2^-60 below the sum of three quarters of the row;
    rounded to 53 bits it would lie above."""
    dev = need_gpu()
    V = 4000
    gen = torch.Generator().manual_seed(V)
    h = ((torch.rand(V // 4, generator=gen) + 0.3) / V).to(dtype)
    h[5] = 2.0 ** -50
    row = torch.cat([h[torch.randperm(V // 4, generator=gen)] for _ in range(4)])
    row[int((row == 2.0 ** -50).nonzero()[1])] = 2.0 ** -50 * (1 + 5 / 64)     # 80 x 2^-60 more
    assert 0.5 < float(row.double().sum()) < 1 and V // 4 <= int((row == 2.0 ** -50 * (1 + 5 / 64)).nonzero()[0]) < V // 2
    got = run_verify(row.expand(3, 1, V).contiguous(), None, torch.zeros(3, 0, dtype=torch.int32),
                     torch.tensor([[0.75], [0.5], [0.25]]), None, dev)
    assert got[0][0, 0].item() == 3 * V // 4 - 1


def test_verify_feeds_commit_len():
    """commit_len goes to kda_decode_multi as it is: the state equals that after the committed tokens alone."""
    dev = need_gpu()
    from kimi_delta_attention_chunked_gb300 import inputs
    n, k, H = 5, 3, 2
    target, draft, tokens, u = dists(n, k, 200, F32, 2, sharp=0.3)
    out, commit = kda.kda_verify_draft(target.to(dev), draft.to(dev), tokens.to(dev), u.to(dev))
    gen = torch.Generator(device=dev).manual_seed(1)
    sets = [inputs.make_qkv_gates(n, H, 64, 64, BF, gen, dev) for _ in range(k + 1)]
    q, kk, v, beta, la = (torch.stack(x, 1).contiguous() for x in zip(*sets))
    S = torch.randn(n, H, 64, 64, generator=gen, device=dev) * 0.02
    got, want = S.clone(), S.clone()
    kda.kda_decode_multi(q, kk, v, la, beta, got, commit_len=commit, want_o=False)
    for i, c in enumerate(commit.tolist()):
        part = want[i:i + 1].clone()
        kda.kda_decode_multi(*(x[i:i + 1, :c].contiguous() for x in (q, kk, v, la, beta)), part, want_o=False)
        want[i] = part[0]
    assert torch.equal(got, want) and len(set(commit.tolist())) > 1


# ------------------------------------------------------------------ together
def test_step_tables_append_attention():
    """One step end to end: pages laid out, keys written, attended over; equal to one call
    over a cache that was filled by hand."""
    dev = need_gpu()
    page, Hq, Hkv, d = 16, 8, 2, 128
    ctx, new = [40, 0, 17, 100], [3, 50, 0, 1]
    c = make(list(zip(ctx, new)), Hq, Hkv, d, page, BF, dev, seed=6, n_extra=0)
    held = [-(-x // page) for x in ctx]
    table = c["table"].clone()
    free = [int(c["table"][n, b]) for n in range(4) for b in range(held[n], -(-(ctx[n] + new[n]) // page))]
    for n in range(4):
        table[n, held[n]:] = -1
    args = on(c, dev)
    table = table.to(dev)
    T = int(c["cu"][-1])
    cu, seq, slot, pos, taken = kda.kda_build_block_tables(i32(ctx, dev), i32(new, dev), i32(free, dev), table, page, T)
    assert torch.equal(table.cpu(), c["table"]) and torch.equal(cu.cpu(), c["cu"]) and torch.equal(seq.cpu(), c["seq"])
    k = args[1].permute(0, 2, 1, 3).reshape(-1, Hkv, d)[slot].contiguous()
    v = args[2].permute(0, 2, 1, 3).reshape(-1, Hkv, d)[slot].contiguous()
    kc, vc = args[1].clone(), args[2].clone()
    kc.permute(0, 2, 1, 3).reshape(-1, Hkv, d)
    for s in slot.tolist():
        kc[s // page, :, s % page] = math.nan
        vc[s // page, :, s % page] = math.nan
    kda.kda_cache_append(k, v, kc, vc, slot)
    assert torch.equal(kc, args[1]) and torch.equal(vc, args[2])
    assert torch.equal(kda.kda_paged_attention(args[0], kc, vc, table, cu, seq), kda.kda_paged_attention(*args))
