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
