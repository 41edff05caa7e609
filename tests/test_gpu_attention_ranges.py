"""Paged attention on the GPU at the ends of fp32: scores past its range, and values that are
not finite at a weight of zero."""
import math

import pytest
import torch

from _gpu import need_gpu
from test_gpu_step import BF, F32, make, on

import kimi_delta_attention_chunked_gb300 as kda

pytestmark = pytest.mark.gpu
FACTORS = [0.125, 4.0, -0.125, -4.0]                       # of the heads' queries


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (BF, 32), (F32, 64)])
@pytest.mark.parametrize("scale", [2.0 ** 127, 2.0 ** 32, 2.0 ** 24])
@pytest.mark.parametrize("ctx,m,falls", [(50, 3, False), (117, 3, False), (20, 1, False), (50, 3, True), (250, 6, True), (200, 300, True)])
def test_attention_large_scales(ctx, m, falls, scale, dtype, d):
    """At these scales the largest score has all the weight (in bf16 a rounded one, and a rounded output); a row whose largest one is past fp32's range (2^29 on
    the tensor cores) is NaN, and does not pass for a row that sees no key.  `falls`: the second half of the keys scores in range."""
    dev = need_gpu()
    gen = torch.Generator().manual_seed(3)
    keys = ctx + m
    rel, most = (2.0 ** -7, 2.0 ** 29) if dtype == BF else (4 * 2.0 ** -24, 2.0 ** 128)
    c = make([(ctx, m)], 4, 1, d, 16, dtype, dev, seed=3)
    b = (128 + torch.randperm(128, generator=gen)[torch.arange(keys) % 128].float()) / 256     # exact in bf16
    if falls:
        b[keys // 2:] *= 2.0 ** -6
    at = c["table"][0].long().repeat_interleave(16)[:keys], torch.arange(keys) % 16
    c["q"].zero_()
    c["q"][..., 0], c["q"][..., 1] = torch.tensor(FACTORS, dtype=dtype), 8.0
    c["k"][at[0], 0, at[1], 0], c["k"][at[0], 0, at[1], 1] = b.to(dtype), 0.0
    values = c["v"][at[0], 0, at[1]].double()
    o, lse = (x.double().cpu() for x in kda.kda_paged_attention(*on(c, dev), scale=scale, want_lse=True))
    b = b.double()
    for t in range(m):
        for h, a in enumerate(FACTORS):
            see = b[:ctx + t + 1]
            j = int((a * see).argmax())
            top = scale * a * float(b[j])
            if abs(top * math.log2(math.e)) >= most:
                assert bool(torch.isnan(o[t, h]).all()) and not math.isfinite(lse[t, h]), (t, h)
            elif int((see == b[j]).sum()) == 1:
                assert bool(((o[t, h] - values[j]).abs() <= rel * values[j].abs()).all()), (t, h)
                assert abs(float(lse[t, h]) - top) <= 4 * 2.0 ** -24 * abs(top), (t, h)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64)])
@pytest.mark.parametrize("n", [1, 200])
def test_attention_infinities_of_no_weight(n, dtype, d):
    """Keys that score -inf in every second tile, with infinite values: 0 * inf makes that channel NaN, in units of one
    CTA as in cut ones; the other channels are as without them."""
    dev = need_gpu()
    c = make([(511, 1)] * n, 4, 4, d, 64, dtype, dev, seed=4)
    c["q"][..., 0] = -1.0
    finite = on(c, dev)
    for r in range(n):
        for lo in (128, 384):
            pages = c["table"][r, lo // 64:lo // 64 + 2].long()
            c["k"][pages, :, :, 0] = math.inf
            c["v"][pages, :, :, 9] = math.inf
    o, lse = (x.double().cpu() for x in kda.kda_paged_attention(*on(c, dev), want_lse=True))
    # the reference: tables without those pages
    finite[3][:, 2:4] = finite[3][:, 6:8] = -1
    ref, rl = (x.double().cpu() for x in kda.kda_paged_attention(*finite, want_lse=True))
    assert not torch.isfinite(o[..., 9]).any()
    keep = torch.arange(d) != 9
    assert torch.allclose(o[..., keep], ref[..., keep], rtol=0, atol=2.0 ** -8 if dtype == BF else 1e-5)
    assert torch.allclose(lse, rl, rtol=0, atol=1e-5)
