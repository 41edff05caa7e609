"""Edges of the serving-step operators on the GPU."""
import pytest
import torch

from _gpu import need_gpu
from test_gpu_step import BF, F32, check, make

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
