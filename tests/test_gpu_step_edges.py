"""Edges of the serving-step operators on the GPU."""
import math

import pytest
import torch

from _gpu import need_gpu
from test_gpu_step import BF, F32, check, make, on

import kimi_delta_attention_chunked_gb300 as kda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (BF, 32), (F32, 64)])
@pytest.mark.parametrize("window", [1, 128, 2 ** 31 - 2, 2 ** 31 - 1])
def test_attention_window_of_rows_before_position_zero(dtype, d, window):
    """More new tokens than the sequence holds, under windows up to the largest: the rows
    at and past position 0 see what they see without the others."""
    dev = need_gpu()
    c = make([(-3, 5), (40, 2), (-200, 201), (-150, 460), (-2, 4), (-7, 7), (0, 3)], 8, 2, d, 16, dtype, dev)
    o, lse = check(c, dev, window=window)
    assert bool((o[:3] == 0).all()) and bool((o[3:5] != 0).any())


def test_verify_negative_draft_probability_counts_as_zero():
    """u q < p with q below 0 and p = 0 would let a token stand that the target never gives."""
    dev = need_gpu()
    for dtype in (F32, BF):
        target = torch.zeros(4, 2, 6, dtype=dtype)
        target[:, :, 1], target[:, :, 2] = 0.25, 0.75
        draft = torch.zeros(4, 1, 6, dtype=dtype)
        draft[:, 0, 1] = 1.0
        tokens = torch.tensor([[5], [5], [2], [1]], dtype=torch.int32)
        draft[0, 0, 5], draft[1, 0, 5], draft[2, 0, 2] = -0.5, -math.inf, -0.5
        u = torch.tensor([[0.5, 0.1], [0.5, 0.1], [0.5, 0.1], [0.5, 0.1]])
        got = kda.kda_verify_draft(target.to(dev), draft.to(dev), tokens.to(dev), u.to(dev))
        # rows 0, 1: p = q = 0, the rest max(p - q, 0) is all on token 2; row 2: stands; row 3: 0.5 < 0.25 fails
        assert got[1].tolist() == [1, 1, 2, 1]
        assert got[0].tolist() == [[2, -1], [2, -1], [2, 1], [2, -1]]
