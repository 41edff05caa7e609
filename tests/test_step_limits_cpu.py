"""Limits and refusals of the serving-step operators that keep every index of
their kernels inside 32 bits and its buffer; nothing here reaches a GPU."""
import pytest
import torch

import kimi_delta_attention_chunked_gb300 as kda
from kimi_delta_attention_chunked_gb300 import _lib as E
from test_step_cpu import P, attention, i32, lib, tables, verify, z  # noqa: F401


@pytest.mark.parametrize("page", [16, 256])
def test_attention_positions_fit_32_bits(lib, page):  # noqa: F811
    """A table that covers 2^31 tokens or next to it: the end of the last key tile would wrap."""
    most = (2 ** 31 - 512) // page
    assert attention(lib, page=page, blocks=most + 1, bytes=0) == E.KDA_ERR_UNSUPPORTED
    assert attention(lib, page=page, blocks=2 ** 31 - 1, bytes=0) == E.KDA_ERR_UNSUPPORTED
    assert attention(lib, page=page, blocks=most, bytes=0) == E.KDA_ERR_WORKSPACE    # accepted up to the next check


def test_verify_vocabulary_fits_32_bits(lib):  # noqa: F811
    """Steps past the end of a row of almost 2^31 numbers would wrap, and read before it."""
    assert verify(lib, V=2 ** 31 - 1, p=None) == E.KDA_ERR_UNSUPPORTED
    assert verify(lib, V=2 ** 30 + 1, p=None) == E.KDA_ERR_UNSUPPORTED
    assert verify(lib, V=2 ** 30, p=None) == E.KDA_ERR_INVALID_ARG      # accepted up to the next check


@pytest.mark.parametrize("kw", [dict(p=P(0x1002)), dict(q=P(0x2001)), dict(dt=E.KDA_BF16, p=P(0x1001)),
                                dict(dt=E.KDA_BF16, q=P(0x2001))])
def test_verify_rows_off_their_elements(lib, kw):  # noqa: F811
    """The rows come as untyped pointers; an element off its own boundary cannot be read."""
    assert verify(lib, **kw) == E.KDA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(seq=P(0x1000)), dict(seq=P(0x2000)), dict(cu=P(0x1000)), dict(pos=P(0x2000)),
                                dict(table=P(0x3000)), dict(taken=P(0x3000)), dict(slot=P(0x1000))])
def test_tables_outputs_over_inputs(lib, kw):  # noqa: F811
    """Lengths updated in place: the CTAs of a step of many tokens would read each other's results."""
    assert tables(lib, **kw) == E.KDA_ERR_INVALID_ARG


def test_binding_want_lse_without_a_truth_value():
    """What its truth value raises is raised, before anything is launched."""
    with pytest.raises(RuntimeError, match="ambiguous"):
        kda.kda_paged_attention(z(5, 4, 32), z(3, 2, 16, 32), z(3, 2, 16, 32), i32(2, 4), i32(3), i32(2), want_lse=z(2))


BIG = 2 ** 32 + 7                                           # 7 when cut to 32 bits


def big(dt, *shape):
    """A tensor of that shape over a single number."""
    return torch.zeros((1,) * len(shape), dtype=dt).expand(*shape)


@pytest.mark.parametrize("call", [
    lambda: kda.kda_build_block_tables(i32(3), i32(3), big(torch.int32, BIG), i32(3, 4), 16, 8),
    lambda: kda.kda_build_block_tables(i32(3), i32(3), i32(4), big(torch.int32, 3, BIG), 16, 8),
    lambda: kda.kda_build_block_tables(big(torch.int32, BIG), big(torch.int32, BIG), i32(4), big(torch.int32, BIG, 4), 16, 8),
    lambda: kda.kda_cache_append(big(torch.float32, BIG, 2, 32), big(torch.float32, BIG, 2, 32), z(3, 2, 16, 32), z(3, 2, 16, 32),
                                 big(torch.int64, BIG)),
    lambda: kda.kda_cache_append(z(5, 2, 32), z(5, 2, 32), big(torch.float32, BIG, 2, 16, 32), big(torch.float32, BIG, 2, 16, 32),
                                 z(5, dt=torch.int64)),
    lambda: kda.kda_paged_attention(big(torch.float32, BIG, 4, 32), z(3, 2, 16, 32), z(3, 2, 16, 32), i32(2, 4), i32(3), i32(2)),
    lambda: kda.kda_paged_attention(z(5, 4, 32), z(3, 2, 16, 32), z(3, 2, 16, 32), big(torch.int32, 2, BIG), i32(3), i32(2)),
    lambda: kda.kda_verify_draft(big(torch.float32, 2, 4, BIG), None, i32(2, 3), z(2, 4)),
    lambda: kda.kda_verify_draft(big(torch.float32, BIG, 1, 9), None, big(torch.int32, BIG, 0), big(torch.float32, BIG, 1)),
])
def test_binding_sizes_are_not_cut_off(call):
    with pytest.raises(ValueError, match="past 2"):
        call()


def test_attention_scale_stays_finite_in_octaves(lib):  # noqa: F811
    """scale log2(e) past the largest float would make NaN of a score of 0."""
    assert attention(lib, scale=2.5e38, bytes=0) == E.KDA_ERR_INVALID_ARG
    assert attention(lib, scale=2.0 ** 127, bytes=0) == E.KDA_ERR_WORKSPACE      # accepted up to the next check
    assert attention(lib, scale=1e-45, bytes=0) == E.KDA_ERR_WORKSPACE
