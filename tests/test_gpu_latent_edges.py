"""Latent attention on the GPU at the ends of its numbers, strides and division."""
import math

import pytest
import torch

import kimi_delta_attention_chunked_gb300 as kda
from _gpu import need_gpu
from _latent import LATENT, NOPE, ROPE, assert_close, expanded_ref, rows_ref
from test_gpu_latent import BF16, DTYPES, FP32, SCALE, absorbed_case, check_expanded, expanded_case, on_gpu, run_absorbed

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    return need_gpu()


def same_kind(got, want, bound, what):
    """`want` within `bound` where it is finite; not finite where it is not."""
    got = got.double().cpu()
    odd = ~torch.isfinite(want)
    assert not torch.isfinite(got[odd]).any(), f"{what}: {int(torch.isfinite(got[odd]).sum())} finite of {int(odd.sum())}"
    assert_close(torch.where(odd, torch.zeros_like(got), got), torch.where(odd, torch.zeros_like(want), want), bound, what)


# ------------------------------------------------------------------ values that are not finite, seen at a weight of zero
# (earlier tokens, new ones) of the requests; the keys of each whose channel becomes infinite
SEEN = {
    "at the edge of one tile": ([(57, 6)], lambda n: [60]),
    "in and behind whole tiles": ([(130, 2)] * 160, lambda n: [10] if n % 3 == 0 else [131] if n % 3 == 1 else []),
    "all keys of a part": ([(5000, 2)], lambda n: list(range(64, 192)) + [5001]),
}


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("where", list(SEEN))
def test_absorbed_infinities_of_no_weight(where, dt):
    """An infinite latent against a query of the other sign scores -inf: its key weighs nothing, and 0 * inf makes
    that channel NaN for the rows that see it, wherever its tile lies and however the keys are divided."""
    lens, odd = SEEN[where]
    H = 3
    q, cache, table, cu, seq = absorbed_case(lens, H, 64, dt, seed=1)
    q[..., 7] = -q[..., 7].abs() - 1.0
    T = q.shape[0]
    o = torch.zeros(T, H, LATENT, dtype=torch.float64)
    lse, bo, bl = torch.zeros(T, H, dtype=torch.float64), torch.zeros_like(o), torch.zeros(T, H, dtype=torch.float64)
    for n, (ctx, m) in enumerate(lens):
        keys, bad = ctx + m, torch.tensor(odd(n), dtype=torch.long)
        rows = cache[table[n].long().repeat_interleave(64)[:keys], torch.arange(keys) % 64].double()
        good = torch.ones(keys, dtype=torch.bool)
        good[bad] = False
        for i in range(m):
            K = rows[:ctx + i + 1][good[:ctx + i + 1]][:, None]
            t = int(cu[n]) + i
            o[t], lse[t], bo[t], bl[t] = rows_ref(q[t].double(), K, K[..., :LATENT], SCALE, dt)
            if bool((bad <= ctx + i).any()):
                o[t, :, 7] = math.nan
        for j in bad.tolist():
            cache[table[n, j // 64], j % 64, 7] = INF
    got, gl = run_absorbed(q, cache, table, cu, seq)
    same_kind(got, o, bo, "o")
    assert bool(torch.isnan(got.cpu()[..., 7][torch.isnan(o[..., 7])]).all())
    assert_close(gl, lse, bl, "lse")


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("lens,keys", [([(40, 60)], [45]), ([(300, 700)], [3, 690]), ([(2, 5000)], list(range(128, 384))),
                                       ([(300, 2000)], list(range(128, 640))), ([(100, 256)], list(range(128, 256)))])
def test_expanded_infinities_of_no_weight(lens, keys, dt):
    """The same of keys that score -inf in the expanded form: the channel is not finite for the rows that see the key,
    the others are as without it."""
    H = 2
    q, kn, kr, v, cu, cu_k = case = expanded_case(lens, H, dt, seed=2)
    q[..., NOPE] = -q[..., NOPE].abs() - 1.0
    (m, s), bad = lens[0], torch.tensor(keys)
    good = torch.ones(s, dtype=torch.bool)
    good[bad] = False
    K = torch.cat([kn, kr[:, None].expand(s, H, ROPE)], 2).double()
    V = v.double()
    o = torch.zeros(m, H, 128, dtype=torch.float64)
    lse, bo, bl = torch.zeros(m, H, dtype=torch.float64), torch.zeros_like(o), torch.zeros(m, H, dtype=torch.float64)
    for i in range(m):
        g = good[:s - m + i + 1]
        o[i], lse[i], bo[i], bl[i] = rows_ref(q[i].double(), K[:len(g)][g], V[:len(g)][g], SCALE, dt)
        if not bool(g.all()):
            o[i, 1, 9] = math.nan
    kr[bad, 0] = INF
    v[bad, 1, 9] = INF
    got, gl = kda.kda_expanded_attention(*on_gpu(case), scale=SCALE, want_lse=True)
    same_kind(got, o, bo, "o")
    assert_close(gl, lse, bl, "lse")


# ------------------------------------------------------------------ scores past the range of fp32
FACTORS = [0.125, 4.0, -0.125, -4.0]                       # of the heads' queries


def sharp(keys, falls, dt, gen):
    """Keys whose first channel has distinct values from 1/2 to 1 in any order, exact in bf16, and 2^-6 of such in the
    second half of the keys if `falls`; the second channel is 0."""
    b = (128 + torch.randperm(128, generator=gen)[torch.arange(keys) % 128].float()) / 256
    if falls:
        b[keys // 2:] *= 2.0 ** -6
    rows = torch.zeros(keys, 2)
    rows[:, 0] = b
    return b.double(), rows.to(dt)


def check_sharp(o, lse, b, values, seen, scale):
    """Row by row.  At these scales (2^24 and more: neighbours are at least 2^-17 2^24 apart, e^-128) the largest score
    has all the weight, in bf16 a rounded one and a rounded output; past fp32's range, or 2^29 on the tensor cores,
    the row is NaN."""
    rel, most = (2.0 ** -7, 2.0 ** 29) if o.dtype == BF16 else (4 * 2.0 ** -24, 2.0 ** 128)
    o, lse = o.double().cpu(), lse.double().cpu()
    for t, n in enumerate(seen):
        for h, a in enumerate(FACTORS):
            j = int((a * b[:n]).argmax())
            top = scale * a * float(b[j])
            if int((b[:n] == b[j]).sum()) > 1:         # two keys share the weight
                continue
            if abs(top * math.log2(math.e)) >= most:
                assert bool(torch.isnan(o[t, h]).all()) and not bool(torch.isfinite(lse[t, h])), (t, h, o[t, h, :4], lse[t, h])
            else:
                want = values(j, h).double()
                assert bool(((o[t, h] - want).abs() <= rel * want.abs()).all()), (t, h)
                assert abs(float(lse[t, h]) - top) <= 4 * 2.0 ** -24 * abs(top), (t, h)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("scale", [2.0 ** 127, 2.0 ** 60, 2.0 ** 32, 2.0 ** 28, 2.0 ** 24])
@pytest.mark.parametrize("ctx,m,falls", [(50, 3, False), (117, 3, False), (20, 1, False), (50, 3, True), (130, 2, True), (250, 6, True)])
def test_absorbed_large_scales(ctx, m, falls, scale, dt):
    gen = torch.Generator().manual_seed(3)
    q, cache, table, cu, seq = absorbed_case([(ctx, m)], len(FACTORS), 16, dt, seed=3)
    b, rows = sharp(ctx + m, falls, dt, gen)
    q.zero_()
    q[..., 0], q[..., 1] = torch.tensor(FACTORS, dtype=dt), 8.0
    at = table[0].long().repeat_interleave(16)[:ctx + m], torch.arange(ctx + m) % 16
    for c in range(2):
        cache[at[0], at[1], c] = rows[:, c]
    flat = cache[at]
    o, lse = run_absorbed(q, cache, table, cu, seq, scale=scale)
    check_sharp(o, lse, b, lambda j, h: flat[j, :LATENT], [ctx + i + 1 for i in range(m)], scale)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("scale", [2.0 ** 127, 2.0 ** 60, 2.0 ** 32, 2.0 ** 28, 2.0 ** 24])
@pytest.mark.parametrize("m,s,falls", [(3, 53, False), (40, 120, False), (1, 100, False), (3, 53, True), (40, 250, True), (300, 600, True)])
def test_expanded_large_scales(m, s, falls, scale, dt):
    gen = torch.Generator().manual_seed(4)
    q, kn, kr, v, cu, cu_k = case = expanded_case([(m, s)], len(FACTORS), dt, seed=4)
    b, rows = sharp(s, falls, dt, gen)
    q.zero_()
    q[..., 0], q[..., 1] = torch.tensor(FACTORS, dtype=dt), 8.0
    kn[..., :2] = rows[:, None]
    o, lse = kda.kda_expanded_attention(*on_gpu(case), scale=scale, want_lse=True)
    check_sharp(o, lse, b, lambda j, h: v[j, h], [s - m + i + 1 for i in range(m)], scale)


# ------------------------------------------------------------------ angles
def test_rotary_small_angles():
    """The sine of a small angle keeps fp32's relative accuracy: half a step of the angle's conversion, sincospi's own
    step, and the frequency's fixed point (2^-64 turns of a position: 2^-30 of the least angle here)."""
    freq = torch.tensor([1e-9, 3.3e-8, 1e-6, 1e-5, 7e-4, 0.02, 0.3, 0.77], dtype=FP32)
    pos = torch.tensor([1, -1, 3, 100], dtype=torch.int32)
    x = torch.zeros(len(pos), 1, 16)
    x[..., :8] = 1.0
    got = kda.kda_rotary(x.cuda(), pos.cuda(), freq.cuda()).double().cpu()
    w = pos.double()[:, None] * freq.double()
    near = w.abs() < 0.78                                  # an eighth of a turn: behind it a quarter is taken off
    err = (got[:, 0, 8:] - w.sin()).abs() / w.sin().abs()
    assert bool((err <= 4 * 2.0 ** -24)[near].all()), err


# ------------------------------------------------------------------ views
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("shared", ["v", "k", "both"])
def test_expanded_heads_share_keys_and_values(shared, dt):
    """One head's keys or values for all of them: views with a head stride of 0."""
    q, kn, kr, v, cu, cu_k = expanded_case([(30, 90), (140, 150)], 4, dt)
    if shared != "v":
        kn = kn[:, :1].expand(-1, 4, -1)
    if shared != "k":
        v = v[:, :1].expand(-1, 4, -1)
    ref, lref, bo, bl = expanded_ref(q, kn, kr, v, cu, cu_k, SCALE, True)
    put = lambda x: x[:, :1].cuda().expand(-1, 4, -1) if x.stride(1) == 0 else x.cuda()  # noqa: E731
    kd, vd = put(kn), put(v)
    assert (kd.stride(1) == 0) == (shared != "v") and (vd.stride(1) == 0) == (shared != "k")
    o, lse = kda.kda_expanded_attention(q.cuda(), kd, kr.cuda(), vd, cu.cuda(), cu_k.cuda(), want_lse=True)
    assert_close(o, ref, bo, "o")
    assert_close(lse, lref, bl, "lse")


# ------------------------------------------------------------------ division
def test_expanded_on_cuda_cores_uses_every_place():
    """300 tiles, each of one place, go to 300 CTAs where so many fit: the unit that CTA 0 begins has as many parts."""
    props = torch.cuda.get_device_properties(0)
    ctas = min(304, 2 * props.multi_processor_count, 300)
    case = on_gpu(expanded_case([(32, 300 * 32)], 1, FP32))
    ws = torch.zeros(kda.kda_expanded_attention_workspace_size(32, 1, FP32), dtype=torch.uint8, device="cuda")
    kda.kda_expanded_attention(*case, causal=False, workspace=ws)
    meta = ws[:32].view(torch.int32).tolist()              # of CTA 0's two slots
    assert meta[4:7] == [0, 0, 32] and meta[7] & 0xffff == ctas


def test_expanded_of_single_row_tiles_uses_every_place():
    """24 key tiles and 5 places for their fixed cost, for 24 pairs: calls of up to 256 tokens have no unit of two steps a
    tile, for which a piece must have two places."""
    if torch.cuda.get_device_properties(0).multi_processor_count < 2 * 29:
        pytest.skip("fewer pairs than places")
    case = on_gpu(expanded_case([(20, 24 * 128)], 1, BF16))
    ws = torch.zeros(kda.kda_expanded_attention_workspace_size(20, 1, BF16), dtype=torch.uint8, device="cuda")
    kda.kda_expanded_attention(*case, causal=False, workspace=ws)
    meta = ws[:2 * 80 * 16].view(torch.int32).view(80, 2, 4)   # of each pair's two slots
    assert meta[5, 1].tolist() == [0, 0, 20, 5 << 16 | 24]


def test_expanded_on_cuda_cores_counts_steps():
    """Two units of 32 tokens and ten tiles each, every tile one place: ten CTAs to either."""
    case = on_gpu(expanded_case([(64, 320)], 1, FP32))
    ws = torch.zeros(kda.kda_expanded_attention_workspace_size(64, 1, FP32), dtype=torch.uint8, device="cuda")
    kda.kda_expanded_attention(*case, causal=False, workspace=ws)
    meta = ws[:2 * 304 * 16].view(torch.int32).view(304, 2, 4)
    assert meta[0, 1].tolist() == [0, 0, 32, 10] and meta[10, 1].tolist() == [32, 0, 32, 10 << 16 | 10]


@pytest.mark.parametrize("lens,H", [([(1500, 9000)], 1), ([(1024, 6000)], 40), ([(256, 6000), (700, 5000)], 24)])
def test_expanded_long_runs_of_tiles(lens, H):
    """Units of dozens of key tiles, in one piece and with borders inside them; a sample of rows and heads is checked."""
    q, kn, kr, v, cu, cu_k = case = expanded_case(lens, H, BF16, seed=H)
    o, lse = kda.kda_expanded_attention(*on_gpu(case), scale=SCALE, want_lse=True)
    o, lse = o.cpu(), lse.cpu()
    gen = torch.Generator().manual_seed(5)
    for n, (m, s) in enumerate(lens):
        t0, k0 = int(cu[n]), int(cu_k[n])
        for i in [0, m - 1] + torch.randint(0, m, (30,), generator=gen).tolist():
            hs = torch.randperm(H, generator=gen)[:3]
            sees = slice(k0, k0 + s - m + i + 1)
            K = torch.cat([kn[sees][:, hs], kr[sees][:, None].expand(-1, len(hs), -1)], 2).double()
            ref, lref, bo, bl = rows_ref(q[t0 + i, hs].double(), K, v[sees][:, hs].double(), SCALE, BF16)
            assert_close(o[t0 + i, hs], ref, bo, f"o of token {i}")
            assert_close(lse[t0 + i, hs], lref, bl, f"lse of token {i}")


@pytest.mark.parametrize("seed", range(16))
def test_expanded_chance_of_few_tokens(seed):
    """Calls of up to 256 tokens over long keys by chance: pieces of one place, borders wherever they fall."""
    import random
    rng = random.Random(500 + seed)
    dt, H, left, lens = rng.choice([BF16, BF16, FP32]), rng.choice([1, 1, 2, 3]), 256, []
    for _ in range(rng.randint(1, 6)):
        m = rng.choice([0, 1, rng.randint(0, 40), rng.randint(0, 250)])
        if m <= left:
            lens.append((m, rng.choice([0, 1, rng.randint(0, 300), rng.randint(0, 3000)])))
            left -= m
    lens.append((left, rng.randint(0, 1500)) if rng.random() < 0.3 else (min(left, 1), 700))
    check_expanded(expanded_case(lens, H, dt, seed=seed), causal=rng.random() < 0.6)
