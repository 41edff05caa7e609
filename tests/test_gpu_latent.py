"""Latent attention on the GPU against plain fp64 forms: rotary positions, the
paged latent cache, absorbed and expanded attention, and a run of them together."""
import pytest
import torch

import kimi_delta_attention_chunked_gb300 as kda
from _gpu import need_gpu
from _latent import absorbed_ref, assert_close, expanded_ref, turned
from _step import lay_out

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
DTYPES = [BF16, FP32]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    return need_gpu()


def rnd(gen, *shape, dt=FP32, scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).to(dt)


# ------------------------------------------------------------------ rotary
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,d,rot", [(1, 1, 2, 2), (3, 2, 64, 64), (7, 5, 128, 64), (33, 3, 96, 32), (5, 4, 30, 14), (2, 1, 256, 256),
                                       (300, 8, 192, 96), (4, 33, 72, 8), (2, 3, 17, 6)])
def test_rotary(T, H, d, rot, interleaved, dt):
    gen = torch.Generator().manual_seed(T + d)
    x = rnd(gen, T, H, d, dt=dt)
    pos = torch.randint(0, 1 << 20, (T,), generator=gen, dtype=torch.int32)
    pos[0] = 0
    freq, _ = kda.rotary_frequencies(rot, device="cpu")
    ref, bound = turned(x, pos, freq, 1.25, interleaved)
    xd = x.cuda()
    got = kda.kda_rotary(xd, pos.cuda(), freq.cuda(), factor=1.25, interleaved=interleaved)
    assert got.data_ptr() != xd.data_ptr() and torch.equal(xd.cpu(), x)
    assert_close(got, ref, bound, "rotary")
    # the same in place, and between views of wider tensors at odd places
    assert kda.kda_rotary(xd, pos.cuda(), freq.cuda(), factor=1.25, interleaved=interleaved, out=xd) is xd
    assert torch.equal(xd, got)
    wide = torch.full((T, H, d + 5), 7.0, dtype=dt).cuda()
    wide[..., 3:3 + d] = x.cuda()
    kda.kda_rotary(wide[..., 3:3 + d], pos.cuda(), freq.cuda(), factor=1.25, interleaved=interleaved, out=wide[..., 3:3 + d])
    assert torch.equal(wide[..., 3:3 + d], got) and bool((wide[..., :3] == 7).all()) and bool((wide[..., 3 + d:] == 7).all())
    turned_about = torch.zeros(H, T, d, dtype=dt).cuda().transpose(0, 1)          # heads before tokens
    kda.kda_rotary(x.cuda(), pos.cuda(), freq.cuda(), factor=1.25, interleaved=interleaved, out=turned_about)
    assert torch.equal(turned_about, got)


def test_rotary_positions():
    """Every int32 position, frequencies from above one to almost none, and one that is not a number."""
    pos = torch.tensor([0, 1, -1, 2, 12345, 999983, 2 ** 24 + 1, 2 ** 30 + 12345, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    freq = torch.tensor([1.0, 6.5, 0.5, 2.0 ** -20, 1e-5, 3e-30, 1e-42, 0.0, -0.75, 0.999999, 1e4 ** -0.5, float("nan")])
    x = torch.zeros(len(pos), 1, 24)
    x[..., 0::2] = 1.0
    got = kda.kda_rotary(x.cuda(), pos.cuda(), freq.cuda(), interleaved=True).double().cpu()
    w = pos.double()[:, None] * freq.double()
    # beyond the roundings of fp32: p 2^-64 turns of the frequency in fixed point, and the check's own
    # product in fp64, off by half a step of the angle
    slack = 8 * 2.0 ** -24 + w.abs() * 2.0 ** -52 + 2.0 ** -30
    assert bool(((got[:, 0, 0::2] - w.cos()).abs() <= slack)[:, :-1].all()) and bool(((got[:, 0, 1::2] - w.sin()).abs() <= slack)[:, :-1].all())
    assert bool(torch.isnan(got[:, 0, -2:]).all())


def test_rotary_nothing():
    x = torch.zeros(0, 4, 64, device="cuda")
    assert kda.kda_rotary(x, torch.zeros(0, dtype=torch.int32, device="cuda"), torch.ones(8, device="cuda")).shape == (0, 4, 64)


def test_rotary_overlapping_output():
    x = torch.zeros(4, 2, 64, device="cuda")
    out = torch.zeros(2, 64, device="cuda").expand(4, 2, 64)
    with pytest.raises(kda.KDAError):
        kda.kda_rotary(x, torch.zeros(4, dtype=torch.int32, device="cuda"), torch.ones(8, device="cuda"), out=out)


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("mode", ["copied", "interleaved", "halves"])
@pytest.mark.parametrize("T,page,odd", [(1, 16, 0), (37, 16, 0), (300, 64, 1), (5, 256, 3), (2000, 32, 0)])
def test_append(T, page, odd, mode, dt):
    gen = torch.Generator().manual_seed(T + page)
    n_pages = -(-T // page) + 3
    both = rnd(gen, T, 640 + odd, dt=dt)
    c, part = both[:, odd:512 + odd], both[:, 512 + odd:576 + odd]
    slot = torch.randperm(n_pages * page, generator=gen)[:T]
    if T > 4:
        slot[1], slot[3] = -1, n_pages * page           # skipped: below the first and past the last
    pos = torch.randint(0, 1 << 20, (T,), generator=gen, dtype=torch.int32)
    freq, _ = kda.rotary_frequencies(64, device="cpu")
    cache = rnd(gen, n_pages, page, 576, dt=dt)
    ref, bound = cache.double().clone().reshape(-1, 576), torch.zeros(n_pages * page, 576, dtype=torch.float64)
    turn, tb = turned(part[:, None], pos, freq, 1.1, mode == "interleaved")
    live = (slot >= 0) & (slot < n_pages * page)
    ref[slot[live], :512] = c[live].double()
    ref[slot[live], 512:] = part[live].double() if mode == "copied" else turn[live, 0]
    if mode != "copied":
        bound[slot[live], 512:] = tb[live, 0]
    bd = both.cuda()
    got = cache.cuda()
    kw = {} if mode == "copied" else dict(positions=pos.cuda(), inv_freq=freq.cuda(), factor=1.1, interleaved=mode == "interleaved")
    kda.kda_latent_append(bd[:, odd:512 + odd], bd[:, 512 + odd:576 + odd], got, slot.cuda(), **kw)
    assert_close(got.reshape(-1, 576), ref, bound, "append")


def test_append_turns_as_rotary_does():
    gen = torch.Generator().manual_seed(3)
    part, pos = rnd(gen, 50, 64, dt=BF16).cuda(), torch.randint(0, 9000, (50,), generator=gen, dtype=torch.int32).cuda()
    freq, _ = kda.rotary_frequencies(64)
    cache = torch.zeros(4, 16, 576, dtype=BF16, device="cuda")
    for inter in (False, True):
        kda.kda_latent_append(torch.zeros(50, 512, dtype=BF16, device="cuda"), part, cache, torch.arange(50, device="cuda"),
                              pos, freq, interleaved=inter)
        assert torch.equal(cache.reshape(-1, 576)[:50, 512:], kda.kda_rotary(part[:, None], pos, freq, interleaved=inter)[:, 0])


# ------------------------------------------------------------------ absorbed
SCALE = 192 ** -0.5


def absorbed_case(lens, H, page, dt, seed=0, extra=3, blocks=None, q_extra=0):
    gen = torch.Generator().manual_seed(seed)
    table, cu, seq, n_pages = lay_out(lens, page, extra, gen, blocks)
    T = int(cu[-1]) + q_extra
    return rnd(gen, T, H, 576, dt=dt), rnd(gen, n_pages, page, 576, dt=dt), table, cu, seq


def run_absorbed(q, cache, table, cu, seq, scale=SCALE, **kw):
    return kda.kda_latent_attention(q.cuda(), cache.cuda(), table.cuda(), cu.cuda(), seq.cuda(), scale, want_lse=True, **kw)


def check_absorbed(q, cache, table, cu, seq, scale=SCALE, given=None):
    """`given`: what the kernel gets in place of the cache (with other values at places that no row sees)."""
    ref, lref, bo, bl = absorbed_ref(q, cache, table, cu, seq, scale)
    o, lse = run_absorbed(q, cache if given is None else given, table, cu, seq, scale)
    assert_close(o, ref, bo, "o")
    assert_close(lse, lref, bl, "lse")
    assert kda.kda_get_last_device_status() == 0
    return o, lse


LENS = {
    "one": [(0, 1)],
    "single tokens": [(0, 1), (15, 1), (16, 1), (63, 1), (127, 1), (128, 1), (500, 1), (1, 1)],
    "verify": [(100, 8), (3, 8), (255, 8), (0, 8)],
    "mixed": [(0, 5), (77, 1), (0, 0), (40, 0), (130, 70), (12, 3), (0, 129)],
    "chunk": [(300, 200)],
}


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("H", [1, 5, 16, 32, 40, 64, 65, 96, 128])
@pytest.mark.parametrize("lens", ["single tokens", "verify"])
def test_absorbed_heads(lens, H, dt):
    check_absorbed(*absorbed_case(LENS[lens], H, 32, dt, seed=H))


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("lens", list(LENS))
def test_absorbed_pages(lens, page, dt):
    check_absorbed(*absorbed_case(LENS[lens], 8, page, dt, seed=page))


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("H", [8, 128])
def test_absorbed_cut_units(H, dt):
    """Few long requests: every unit is shared by many CTAs and joined."""
    check_absorbed(*absorbed_case([(3001, 1), (4000, 2)], H, 64, dt, seed=H))


@pytest.mark.parametrize("dt", DTYPES)
def test_absorbed_many_requests(dt):
    check_absorbed(*absorbed_case([(17 * i % 301, 1 + i % 3) for i in range(400)], 4, 16, dt))


def test_thousands_of_requests():
    """More requests than one warp looks through alone."""
    check_absorbed(*absorbed_case([(7 * i % 90, i % 3) for i in range(1500)], 2, 16, BF16))
    check_expanded(expanded_case([(i % 4, 5 * i % 70) for i in range(1300)], 1, BF16))


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("bad", [-1, "n_pages", 2 ** 31 - 1, -2 ** 31])
def test_absorbed_missing_pages(bad, dt):
    q, cache, table, cu, seq = absorbed_case([(100, 4), (300, 1), (0, 3), (20, 2)], 16, 16, dt)
    bad = cache.shape[0] if bad == "n_pages" else bad
    for n, b in ((0, 2), (1, 0), (1, 9), (1, 18), (2, 0), (3, 1)):
        table[n, b] = bad
    check_absorbed(q, cache, table, cu, seq)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("odd", [float("nan"), float("inf"), -float("inf"), "lowest"])
def test_absorbed_unseen_places(odd, dt):
    """What stands behind the last token, in other pages, and in the rows of later new tokens reaches no row that
    does not see it."""
    lens = [(100, 4), (300, 1), (0, 3), (127, 2), (0, 70), (5, 0)]
    for H in (3, 32, 128):
        q, cache, table, cu, seq = absorbed_case(lens, H, 64, dt, seed=H)
        value = torch.finfo(dt).min if odd == "lowest" else odd
        given = torch.full_like(cache, value)
        for n in range(len(lens)):
            for j in range(int(seq[n])):
                given[table[n, j // 64], j % 64] = cache[table[n, j // 64], j % 64]
        check_absorbed(q, cache, table, cu, seq, given=given)
        # the last new token's own row: only that token may be affected
        last = [(n, int(seq[n]) - 1) for n, (_, m) in enumerate(lens) if m > 1]
        for n, j in last:
            given[table[n, j // 64], j % 64] = value
        ref, lref, bo, bl = absorbed_ref(q, cache, table, cu, seq, SCALE)
        o, lse = run_absorbed(q, given, table, cu, seq)
        for n, _ in last:
            bo[int(cu[n + 1]) - 1] = bl[int(cu[n + 1]) - 1] = float("inf")
        assert_close(o, ref, bo, "o")
        assert_close(lse, lref, bl, "lse")


@pytest.mark.parametrize("dt", DTYPES)
def test_absorbed_seen_infinities(dt):
    """An infinite latent channel reaches exactly the rows that see it."""
    q, cache, table, cu, seq = absorbed_case([(60, 6), (200, 3)], 40, 16, dt)
    q[:, :, 7] = 0.0
    n, j = 0, 62
    cache[table[n, j // 16], j % 16, 7] = float("inf")
    o, lse = run_absorbed(q, cache, table, cu, seq)
    # 0 * inf makes the score NaN: rows from position 62 on are NaN, the ones before it are as without it
    clean = cache.clone()
    clean[table[n, j // 16], j % 16, 7] = 0.0
    ref, lref, bo, bl = absorbed_ref(q, clean, table, cu, seq, SCALE)
    bo[2:6], bl[2:6] = float("inf"), float("inf")
    assert_close(o, ref, bo, "o")
    assert_close(lse, lref, bl, "lse")
    assert bool(torch.isnan(lse[2:6]).all()) and bool(torch.isnan(o[2:6]).all())


@pytest.mark.parametrize("dt", DTYPES)
def test_absorbed_padding_and_reuse(dt):
    """Rows behind the last request stay as they were; buffers passed in are the ones returned; lse is optional."""
    q, cache, table, cu, seq = absorbed_case([(9, 2), (0, 0), (40, 1)], 20, 16, dt, q_extra=5)
    ref, lref, bo, bl = absorbed_ref(q, cache, table, cu, seq, SCALE)
    o = torch.full((8, 20, 512), 3.0, dtype=dt, device="cuda")
    lse = torch.full((8, 20), 5.0, device="cuda")
    ws = torch.empty(kda.kda_latent_attention_workspace_size(8, 20, dt), dtype=torch.uint8, device="cuda")
    a, b = run_absorbed(q, cache, table, cu, seq, o=o, lse=lse, workspace=ws)
    assert a is o and b is lse
    assert_close(o, ref, bo, "o")
    assert_close(lse, lref, bl, "lse")
    assert bool((o[3:] == 3).all()) and bool((lse[3:] == 5).all())
    alone = kda.kda_latent_attention(q.cuda(), cache.cuda(), table.cuda(), cu.cuda(), seq.cuda(), SCALE)
    assert torch.equal(alone[:3], o[:3])


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("gap", [8, 3])
def test_absorbed_strided_queries(gap, dt):
    """Tokens of q further apart than they are long; at 3 elements more, off 16-byte boundaries."""
    q, cache, table, cu, seq = absorbed_case([(50, 3), (7, 1)], 6, 16, dt)
    wide = torch.zeros(4, 6 * 576 + gap, dtype=dt).cuda()
    wide[:, :6 * 576] = q.reshape(4, -1).cuda()
    view = wide[:, :6 * 576].unflatten(1, (6, 576))
    o, lse = kda.kda_latent_attention(view, cache.cuda(), table.cuda(), cu.cuda(), seq.cuda(), SCALE, want_lse=True)
    ref, lref, bo, bl = absorbed_ref(q, cache, table, cu, seq, SCALE)
    assert_close(o, ref, bo, "o")
    assert_close(lse, lref, bl, "lse")


@pytest.mark.parametrize("dt", DTYPES)
def test_absorbed_short_tables(dt):
    """Keys past max_blocks * page_size are left out; lengths beyond the table and negative ones stay inside."""
    q, cache, table, cu, seq = absorbed_case([(100, 4), (300, 2)], 8, 16, dt)
    table = table[:, :5].contiguous()
    check_absorbed(q, cache, table, cu, seq)
    # nothing to see at all: no pages, no blocks, a length below the new tokens'
    o, lse = run_absorbed(q, cache, torch.zeros(2, 0, dtype=torch.int32), cu, seq)
    assert not o.any() and bool((lse == -float("inf")).all())
    o, lse = run_absorbed(q, cache[:0], table, cu, seq)
    assert not o.any() and bool((lse == -float("inf")).all())
    check_absorbed(q, cache, table, cu, torch.tensor([2, 0], dtype=torch.int32))
    o, lse = run_absorbed(q, cache, table, cu, torch.tensor([-7, 2 ** 31 - 1], dtype=torch.int32))
    ref, lref, bo, bl = absorbed_ref(q, cache, table, cu, torch.tensor([0, 2 ** 31 - 1], dtype=torch.int32), SCALE)
    assert_close(o, ref, bo, "o")


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("amp", [30.0, 1e-4])
def test_absorbed_sharp_and_flat(amp, dt):
    """Scores that jump by hundreds of octaves from key to key, and ones that hardly differ."""
    q, cache, table, cu, seq = absorbed_case([(700, 3), (260, 1)], 12, 32, dt)
    check_absorbed((q.float() * amp).to(dt), cache, table, cu, seq)


@pytest.mark.parametrize("dt", DTYPES)
def test_absorbed_rising_scores(dt):
    """Each key tile's scores exceed the ones before: the running reference moves at every tile."""
    q, cache, table, cu, seq = absorbed_case([(1500, 2)], 33, 64, dt)
    ramp = torch.arange(1502, dtype=torch.float32) * 0.05
    q[..., 0] = 8.0
    for j in range(1502):
        cache[table[0, j // 64], j % 64, 0] = ramp[j]
    check_absorbed(q, cache, table, cu, seq)


def test_absorbed_captured():
    """A captured call serves other lengths and other inputs when it is replayed; two graphs with a workspace each."""
    q, cache, table, cu, seq = absorbed_case([(300, 2), (40, 1), (0, 4)], 32, 32, BF16, extra=40)
    d = [x.cuda() for x in (q, cache, table, cu, seq)]
    kda.kda_latent_attention(*d, SCALE)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = kda.kda_latent_attention(*d, SCALE, want_lse=True)
        graphs.append((g, out))
    for new_seq, new_cu in ((seq, cu), (torch.tensor([17, 30, 2], dtype=torch.int32), torch.tensor([0, 0, 3, 5], dtype=torch.int32))):
        d[4].copy_(new_seq)
        d[3].copy_(new_cu)
        d[0].copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(5)).to(BF16))
        ref, lref, bo, bl = absorbed_ref(d[0].cpu(), cache, table, new_cu, new_seq, SCALE)
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, (o, lse) in graphs:
            assert_close(o, ref, bo, "o")
            assert_close(lse, lref, bl, "lse")


def test_absorbed_two_streams():
    cases = [absorbed_case([(400 + 50 * i, 3), (20, 1)], 32, 32, BF16, seed=i) for i in range(2)]
    dev = [[x.cuda() for x in c] for c in cases]
    want = [kda.kda_latent_attention(*c, SCALE) for c in dev]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[] for _ in range(2)]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(kda.kda_latent_attention(*dev[i], SCALE, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


# ------------------------------------------------------------------ expanded
def expanded_case(lens, H, dt, seed=0, q_extra=0, k_extra=0, pad=0):
    """lens: (new tokens, keys) of each request; `pad` elements between the rows of the projection."""
    gen = torch.Generator().manual_seed(seed)
    cu = torch.tensor([0] + [a for a, _ in lens]).cumsum(0).to(torch.int32)
    cu_k = torch.tensor([0] + [b for _, b in lens]).cumsum(0).to(torch.int32)
    T, S = int(cu[-1]) + q_extra, int(cu_k[-1]) + k_extra
    both = rnd(gen, S, H, 256 + pad, dt=dt)
    return rnd(gen, T, H, 192, dt=dt), both[..., :128], rnd(gen, S, 64, dt=dt), both[..., 128:256], cu, cu_k


def on_gpu(case):
    """The case on the GPU, views kept as they are."""
    q, kn, kr, v, cu, cu_k = case
    base = kn._base if kn._base is not None and kn._base.shape == (*kn.shape[:2], kn.stride(1)) else None
    if base is None:
        return [x.cuda() for x in case]
    both = base.cuda()
    off = v.storage_offset() - kn.storage_offset()
    return [q.cuda(), both[..., :128], kr.cuda(), both[..., off:off + 128], cu.cuda(), cu_k.cuda()]


def check_expanded(case, causal=True, scale=SCALE, given=None):
    ref, lref, bo, bl = expanded_ref(*case, scale, causal)
    o, lse = kda.kda_expanded_attention(*on_gpu(case if given is None else given), scale=scale, causal=causal, want_lse=True)
    assert_close(o, ref, bo, "o")
    assert_close(lse, lref, bl, "lse")
    assert kda.kda_get_last_device_status() == 0
    return o, lse


KLENS = {
    "one": [(1, 1)],
    "squares": [(1, 1), (127, 127), (128, 128), (129, 129), (2, 2), (64, 64)],
    "context": [(1, 500), (30, 131), (200, 333), (5, 128), (256, 257)],
    "short keys": [(10, 4), (300, 100), (7, 0), (0, 9), (0, 0), (3, 3)],
    "long": [(700, 900)],
}


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens", list(KLENS))
def test_expanded_lengths(lens, causal, dt):
    check_expanded(expanded_case(KLENS[lens], 3, dt), causal)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("H", [1, 2, 16, 40])
def test_expanded_heads(H, dt):
    check_expanded(expanded_case([(70, 90), (3, 200), (130, 130)], H, dt, seed=H))


@pytest.mark.parametrize("dt", DTYPES)
def test_expanded_cut_units(dt):
    """One head and many keys: each unit is shared by many CTAs."""
    check_expanded(expanded_case([(20, 9000)], 1, dt))


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("odd", [float("nan"), float("inf"), "lowest"])
def test_expanded_unseen_places(odd, causal, dt):
    """Keys and values behind a request's end (the next one's, and behind the last) and, causal, of later tokens."""
    lens = [(50, 77), (140, 140), (3, 130), (1, 20)]
    case = expanded_case(lens, 2, dt, k_extra=9)
    q, kn, kr, v, cu, cu_k = case
    value = torch.finfo(dt).min if odd == "lowest" else odd
    ref, lref, bo, bl = expanded_ref(*case, SCALE, causal)
    both, kr2 = kn._base.clone(), kr.clone()
    both[int(cu_k[-1]):], kr2[int(cu_k[-1]):] = value, value
    both[int(cu_k[2]):int(cu_k[3])], kr2[int(cu_k[2]):int(cu_k[3])] = value, value       # all of request 2
    bo[int(cu[2]):int(cu[3])] = bl[int(cu[2]):int(cu[3])] = float("inf")
    if causal:                                                                             # the last tokens' own
        for n in (0, 1):
            both[int(cu_k[n + 1]) - 1], kr2[int(cu_k[n + 1]) - 1] = value, value
            bo[int(cu[n + 1]) - 1] = bl[int(cu[n + 1]) - 1] = float("inf")
    given = (q, both[..., :128], kr2, both[..., 128:256], cu, cu_k)
    o, lse = kda.kda_expanded_attention(*on_gpu(given), scale=SCALE, causal=causal, want_lse=True)
    assert_close(o, ref, bo, "o")
    assert_close(lse, lref, bl, "lse")


@pytest.mark.parametrize("dt", DTYPES)
def test_expanded_seen_infinities(dt):
    """An infinite value in one channel reaches exactly the rows that see it, in that channel."""
    case = expanded_case([(40, 60), (200, 200)], 2, dt)
    q, kn, kr, v, cu, cu_k = case
    ref, lref, bo, bl = expanded_ref(*case, SCALE, True)
    v[45, 1, 9] = float("inf")                              # key 45 of request 0: tokens 25 .. 39 see it
    v[60 + 150, 0, 100] = -float("inf")                     # key 150 of request 1
    v[60 + 150, 0, 3] = float("nan")
    o, lse = kda.kda_expanded_attention(*on_gpu(case), scale=SCALE, want_lse=True)
    want = ref.clone()
    want[25:40, 1, 9] = float("inf")
    want[40 + 150:, 0, 100] = -float("inf")
    assert bool(torch.isnan(o[40 + 150:, 0, 3]).all())
    bo[40 + 150:, 0, 3] = float("inf")
    assert_close(o, want, bo, "o")
    assert_close(lse, lref, bl, "lse")


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("kind", ["packed", "padded", "odd", "head first"])
def test_expanded_layouts(kind, dt):
    """Views: a gap between the heads (of 16 bytes, or of one element), tensors of their own, heads before tokens."""
    case = expanded_case([(30, 90), (140, 150)], 4, dt, pad=8 if kind == "padded" else 1 if kind == "odd" else 0)
    q, kn, kr, v, cu, cu_k = case
    ref, lref, bo, bl = expanded_ref(*case, SCALE, True)
    dev = on_gpu(case)
    if kind == "packed":
        dev[1], dev[3] = dev[1].contiguous(), dev[3].contiguous()
    if kind == "head first":
        dev[1], dev[3] = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (dev[1], dev[3]))
    o, lse = kda.kda_expanded_attention(*dev, scale=SCALE, want_lse=True)
    assert_close(o, ref, bo, "o")
    assert_close(lse, lref, bl, "lse")


@pytest.mark.parametrize("dt", DTYPES)
def test_expanded_padding_and_reuse(dt):
    case = expanded_case([(5, 9), (3, 3)], 6, dt, q_extra=4, k_extra=2)
    ref, lref, bo, bl = expanded_ref(*case, SCALE, True)
    o, lse = torch.full((12, 6, 128), 3.0, dtype=dt, device="cuda"), torch.full((12, 6), 5.0, device="cuda")
    ws = torch.empty(kda.kda_expanded_attention_workspace_size(12, 6, dt), dtype=torch.uint8, device="cuda")
    a, b = kda.kda_expanded_attention(*on_gpu(case), o=o, lse=lse, workspace=ws)
    assert a is o and b is lse
    assert_close(o, ref, bo, "o")
    assert_close(lse, lref, bl, "lse")
    assert bool((o[8:] == 3).all()) and bool((lse[8:] == 5).all())
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    o, lse = kda.kda_expanded_attention(case[0].cuda(), *(x[:0].cuda() for x in case[1:4]), case[4].cuda(), none, want_lse=True)
    assert not o[:8].any() and bool((lse[:8] == -float("inf")).all())       # no keys at all


@pytest.mark.parametrize("dt", DTYPES)
def test_expanded_bad_offsets(dt):
    """Offsets past the tensors are brought inside them."""
    case = list(expanded_case([(20, 30), (10, 40)], 2, dt))
    good = on_gpu(case)
    want = kda.kda_expanded_attention(*good)
    good[4] = torch.tensor([0, 20, 2 ** 31 - 1], dtype=torch.int32).cuda()
    good[5] = torch.tensor([-5, 30, 1000], dtype=torch.int32).cuda()
    assert torch.equal(kda.kda_expanded_attention(*good), want)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("amp", [30.0, 1e-4])
def test_expanded_sharp_and_flat(amp, dt):
    q, *rest = expanded_case([(150, 700), (260, 260)], 2, dt)
    check_expanded(((q.float() * amp).to(dt), *rest))


def test_expanded_captured():
    case = expanded_case([(30, 50), (200, 300)], 4, BF16)
    d = on_gpu(case)
    kda.kda_expanded_attention(*d)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = kda.kda_expanded_attention(*d, want_lse=True)
    for cu, cu_k in ((case[4], case[5]), (torch.tensor([0, 100, 230]), torch.tensor([0, 140, 350]))):
        d[4].copy_(cu.to(torch.int32))
        d[5].copy_(cu_k.to(torch.int32))
        g.replay()
        torch.cuda.synchronize()
        ref, lref, bo, bl = expanded_ref(*case[:4], cu, cu_k, SCALE, True)
        assert_close(o, ref, bo, "o")
        assert_close(lse, lref, bl, "lse")


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("dt", DTYPES)
def test_forms_agree(dt):
    """A layer's two forms on one prompt: tables, rotary, append and absorbed attention against projections and
    expanded attention in two halves that are joined by their lse."""
    gen = torch.Generator().manual_seed(11)
    H, n, page = 4, [70, 33], 16
    T = sum(n)
    c, part = rnd(gen, T, 512, dt=dt).cuda(), rnd(gen, T, 64, dt=dt).cuda()
    q = rnd(gen, T, H, 192, dt=dt).cuda()
    up_k, up_v = rnd(gen, H, 512, 128, scale=512 ** -0.5).cuda(), rnd(gen, H, 512, 128, scale=512 ** -0.5).cuda()
    new = torch.tensor(n, dtype=torch.int32).cuda()
    table = torch.full((2, 5), -1, dtype=torch.int32).cuda()
    cu, seq, slot, pos, _ = kda.kda_build_block_tables(torch.zeros_like(new), new, torch.arange(12, dtype=torch.int32).cuda(), table,
                                                       page, T)
    freq, factor = kda.rotary_frequencies(64, scaling="yarn", scale=4.0)
    q_rope = kda.kda_rotary(q[..., 128:], pos, freq, factor=factor)
    cache = torch.zeros(12, page, 576, dtype=dt, device="cuda")
    kda.kda_latent_append(c, part, cache, slot, pos, freq, factor=factor)
    q_abs = torch.empty(T, H, 576, dtype=dt, device="cuda")
    q_abs[..., :512] = torch.einsum("thd,hcd->thc", q[..., :128].double(), up_k.double()).to(dt)
    q_abs[..., 512:] = q_rope
    latent, lse = kda.kda_latent_attention(q_abs, cache, table, cu, seq, SCALE, want_lse=True)
    absorbed = torch.einsum("thc,hcd->thd", latent.double(), up_v.double())
    # expanded: the last half of each prompt over all of it, in two parts
    k = torch.einsum("tc,hcd->thd", c.double(), up_k.double()).to(dt)
    v = torch.einsum("tc,hcd->thd", c.double(), up_v.double()).to(dt)
    kr = kda.kda_rotary(part[:, None], pos, freq, factor=factor)[:, 0]
    qe = torch.cat([q[..., :128], q_rope], -1)
    halves = [(a, a + m // 2, a + m) for a, m in ((0, n[0]), (n[0], n[1]))]
    tail = torch.cat([torch.arange(b, e) for _, b, e in halves]).cuda()
    head = torch.cat([torch.arange(a, b) for a, b, _ in halves]).cuda()
    offs = lambda xs: torch.tensor([0, *xs]).cumsum(0).to(torch.int32).cuda()  # noqa: E731
    cu_t, cu_h = offs([e - b for _, b, e in halves]), offs([b - a for a, b, _ in halves])
    o1, l1 = kda.kda_expanded_attention(qe[tail], k[tail], kr[tail], v[tail], cu_t, cu_t, want_lse=True)
    o2, l2 = kda.kda_expanded_attention(qe[tail], k[head], kr[head], v[head], cu_t, cu_h, causal=False, want_lse=True)
    joint = torch.logaddexp(l1.double(), l2.double())
    expanded = o1.double() * torch.exp(l1.double() - joint)[..., None] + o2.double() * torch.exp(l2.double() - joint)[..., None]
    # What the forms round differently to the storage type: of a score, q, k and the absorbed q (half a
    # step of each product's magnitude), and the sums of 576 products in fp32; of an output the same in the
    # weights, twice, and the values and latent sums.
    half = 2.0 ** -8 if dt == BF16 else 2.0 ** -24
    mag = SCALE * float(torch.einsum("thc,sc->ths", q_abs.double().abs(), cache.reshape(-1, 576).double().abs()).max())
    ds = mag * (3 * half + 580 * 2.0 ** -24)
    assert float((lse[tail].double() - joint).abs().max()) < 2 * ds
    assert float((absorbed[tail] - expanded).abs().max()) < (4 * ds + 4 * half) * float(v.abs().max())


# ------------------------------------------------------------------ chance sizes, long offsets, order of calls
@pytest.mark.parametrize("seed", range(16))
def test_absorbed_chance(seed):
    """Lengths, heads and pages by chance: units of every kind, cut wherever the division puts its borders."""
    import random
    rng = random.Random(seed)
    dt = rng.choice([BF16, BF16, BF16, FP32])
    H, page, n = rng.choice([1, 2, 3, 7, 16, 33, 48, 64, 100, 128, 129, 200]), rng.choice([16, 32, 64, 128, 256]), rng.randint(1, 40)
    lens = [(rng.choice([0, 1, rng.randint(0, 900)]), rng.choice([0, 1, 1, 1, 2, rng.randint(0, 12)])) for _ in range(n)]
    if sum(m for _, m in lens) == 0:
        lens.append((5, 1))
    check_absorbed(*absorbed_case(lens, H, page, dt, seed=seed))


@pytest.mark.parametrize("seed", range(16))
def test_expanded_chance(seed):
    import random
    rng = random.Random(100 + seed)
    dt, H, n = rng.choice([BF16, BF16, BF16, FP32]), rng.choice([1, 1, 2, 3, 5]), rng.randint(1, 12)
    lens = [(rng.choice([0, 1, 255, 256, 257, 512, 513, rng.randint(0, 700)]), rng.choice([0, 1, rng.randint(0, 300), rng.randint(0, 900)]))
            for _ in range(n)]
    if sum(m for m, _ in lens) == 0:
        lens.append((5, 1))
    check_expanded(expanded_case(lens, H, dt, seed=seed), causal=rng.random() < 0.6)


@pytest.mark.parametrize("tokens", [1, 257, 513])
@pytest.mark.parametrize("keys", [1, 2, 129, 300])
def test_expanded_few_places(tokens, keys):
    """Fewer tiles than CTAs, with row tiles that take one place and two."""
    for n in (1, 3):
        check_expanded(expanded_case([(tokens, keys)] * n, 1, BF16, seed=tokens + keys), causal=False)


@pytest.mark.parametrize("dt", DTYPES)
def test_offsets_past_32_bits(dt):
    """A cache of more than 2^32 bytes and 2^31 elements with the pages of a request at its end."""
    page, n_pages = 256, 16000                          # 2.36e9 channels
    gen = torch.Generator().manual_seed(0)
    small = rnd(gen, 3, page, 576, dt=dt)
    cache = torch.zeros(n_pages, page, 576, dtype=dt, device="cuda")
    q = rnd(gen, 2, 8, 576, dt=dt)
    table, cu, seq = torch.tensor([[2, 0, 1]], dtype=torch.int32), torch.tensor([0, 2], dtype=torch.int32), torch.tensor([600], dtype=torch.int32)
    ref, lref, bo, bl = absorbed_ref(q, small, table, cu, seq, SCALE)
    slot = torch.arange(3 * page, device="cuda") + (n_pages - 3) * page
    rows = small.reshape(-1, 576).cuda()
    kda.kda_latent_append(rows[:, :512], rows[:, 512:], cache, slot)
    assert torch.equal(cache[-3:].cpu(), small) and not cache[:-3].any()
    o, lse = run_absorbed(q, cache, table + (n_pages - 3), cu, seq)
    assert_close(o, ref, bo, "o")
    assert_close(lse, lref, bl, "lse")


def test_expanded_strides_past_32_bits():
    """Tokens of the keys 2^24 elements apart: their offsets pass 2^31."""
    case = expanded_case([(40, 150)], 2, BF16)
    ref, lref, bo, bl = expanded_ref(*case, SCALE, True)
    q, kn, kr, v, cu, cu_k = on_gpu(case)
    far = torch.empty(150 * (1 << 24), dtype=BF16, device="cuda")
    view = far.as_strided((150, 2, 256), (1 << 24, 256, 1))
    view[..., :128], view[..., 128:] = kn, v
    o, lse = kda.kda_expanded_attention(q, view[..., :128], kr, view[..., 128:], cu, cu_k, want_lse=True)
    assert_close(o, ref, bo, "o")
    assert_close(lse, lref, bl, "lse")


def test_rotary_strides_past_32_bits():
    gen = torch.Generator().manual_seed(1)
    x, pos = rnd(gen, 200, 2, 64, dt=BF16), torch.arange(200, dtype=torch.int32)
    freq, _ = kda.rotary_frequencies(64, device="cpu")
    ref, bound = turned(x, pos, freq, 1.0, False)
    far = torch.empty(200 * (1 << 24), dtype=BF16, device="cuda").as_strided((200, 2, 64), (1 << 24, 64, 1))
    far.copy_(x.cuda())
    assert_close(kda.kda_rotary(far, pos.cuda(), freq.cuda(), out=far), ref, bound, "rotary")


def test_calls_in_a_row_share_a_workspace():
    """Calls of both forms one behind the other on one stream, with one workspace and other inputs each time."""
    size = max(kda.kda_latent_attention_workspace_size(4, 32, BF16), kda.kda_expanded_attention_workspace_size(60, 2, BF16))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    a = [[x.cuda() for x in absorbed_case([(300 * i, 2), (50, 1)], 32, 32, BF16, seed=i)] for i in range(4)]
    e = [on_gpu(expanded_case([(30, 400 * i), (20, 20)], 2, BF16, seed=i)) for i in range(4)]
    want_a, want_e = [kda.kda_latent_attention(*c, SCALE) for c in a], [kda.kda_expanded_attention(*c) for c in e]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [(kda.kda_latent_attention(*a[i], SCALE, workspace=ws), kda.kda_expanded_attention(*e[i], workspace=ws)) for i in range(4)]
        torch.cuda.synchronize()
        for i in range(4):
            assert torch.equal(got[i][0], want_a[i]) and torch.equal(got[i][1], want_e[i])


def test_other_stream():
    """A call on another stream than the current one; what it makes is that stream's memory."""
    gen = torch.Generator().manual_seed(2)
    x, pos = rnd(gen, 500, 4, 64, dt=BF16).cuda(), torch.arange(500, dtype=torch.int32, device="cuda")
    freq, _ = kda.rotary_frequencies(64)
    case = on_gpu(expanded_case([(200, 300)], 4, BF16))
    want, want_o = kda.kda_rotary(x, pos, freq), kda.kda_expanded_attention(*case)
    cache, none = torch.zeros(40, 16, 576, dtype=BF16, device="cuda"), torch.zeros(500, 512, dtype=BF16, device="cuda")
    at = torch.arange(500, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        got, got_o = kda.kda_rotary(x, pos, freq, stream=s), kda.kda_expanded_attention(*case, stream=s)
        kda.kda_latent_append(none, x[:, 0], cache, at, pos, freq, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(got, want) and torch.equal(got_o, want_o)
        assert torch.equal(cache.reshape(-1, 576)[:500, 512:], want[:, 0])
        s.wait_stream(torch.cuda.current_stream())


@pytest.mark.parametrize("dt", DTYPES)
def test_append_slot_named_twice(dt):
    """Each piece of the slot's row is one of the two rows'."""
    rows = torch.arange(1, 3, dtype=torch.float32)[:, None].expand(2, 576).to(dt).cuda()
    cache = torch.zeros(1, 16, 576, dtype=dt, device="cuda")
    kda.kda_latent_append(rows[:, :512], rows[:, 512:], cache, torch.tensor([5, 5], device="cuda"))
    got = cache[0, 5].float()
    assert bool(((got == 1) | (got == 2)).all()) and not cache[0, :5].any() and not cache[0, 6:].any()


@pytest.mark.parametrize("H", [257, 700])
def test_absorbed_hundreds_of_heads(H):
    """More heads than one unit holds, and a last group with fewer of them."""
    check_absorbed(*absorbed_case([(150, 2), (0, 1), (333, 1)], H, 64, BF16, seed=H))


def test_two_threads():
    """Calls at once from two host threads, each on its own stream."""
    import threading
    cases = [[x.cuda() for x in absorbed_case([(500 + 90 * i, 2), (33, 1)], 16, 32, BF16, seed=i)] for i in range(2)]
    packed = [on_gpu(expanded_case([(150, 300 + 70 * i), (5, 9)], 3, BF16, seed=i)) for i in range(2)]
    want = [(kda.kda_latent_attention(*cases[i], SCALE), kda.kda_expanded_attention(*packed[i])) for i in range(2)]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(25):
                got = kda.kda_latent_attention(*cases[i], SCALE), kda.kda_expanded_attention(*packed[i])
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    assert kda.kda_get_last_device_status() == 0


def test_absorbed_beside_other_kernels():
    """On another stream the recurrent layer's prefill holds shared memory and TMEM of the same SMs."""
    from kimi_delta_attention_chunked_gb300 import inputs
    w = inputs.Workload("beside", "prefill", H=32, dk=128, dv=128, dtype=BF16, chunk=64)
    d = inputs.make_prefill(w, device=torch.device("cuda", 0), seed=0, lengths=[2048])
    run = lambda: kda.kda_prefill(d["q"], d["k"], d["v"], d["log_alpha"], d["beta"], cu_seqlens=d["cu_seqlens"],  # noqa: E731
                                  cu_seqlens_host=d["cu_seqlens_host"], chunk=64)
    case = [x.cuda() for x in absorbed_case([(2000, 1), (700, 3)], 32, 64, BF16)]
    packed = on_gpu(expanded_case([(600, 900)], 4, BF16))
    want, want_e, want_p = kda.kda_latent_attention(*case, SCALE), kda.kda_expanded_attention(*packed), run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(10):
        with torch.cuda.stream(side):
            got_p = [run() for _ in range(3)]
        got = [(kda.kda_latent_attention(*case, SCALE), kda.kda_expanded_attention(*packed)) for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, want) and torch.equal(b, want_e) for a, b in got)
        assert all(torch.equal(a[0], want_p[0]) and torch.equal(a[1], want_p[1]) for a in got_p)
