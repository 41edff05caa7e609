"""Limits and refusals of the serving-step operators that keep every index of
their kernels inside 32 bits and its buffer; nothing here reaches a GPU."""
import pytest

from kimi_delta_attention_chunked_gb300 import _lib as E
from test_step_cpu import P, attention, lib  # noqa: F401


@pytest.mark.parametrize("page", [16, 256])
def test_attention_positions_fit_32_bits(lib, page):  # noqa: F811
    """A table that covers 2^31 tokens or next to it: the end of the last key tile would wrap."""
    most = (2 ** 31 - 512) // page
    assert attention(lib, page=page, blocks=most + 1, bytes=0) == E.KDA_ERR_UNSUPPORTED
    assert attention(lib, page=page, blocks=2 ** 31 - 1, bytes=0) == E.KDA_ERR_UNSUPPORTED
    assert attention(lib, page=page, blocks=most, bytes=0) == E.KDA_ERR_WORKSPACE    # accepted up to the next check
