"""Strides that the latent-attention operators take and refuse, before anything reaches a GPU."""
import pytest

from kimi_delta_attention_chunked_gb300 import _lib as E
from test_latent_cpu import expanded
from test_step_cpu import lib  # noqa: F401


@pytest.mark.parametrize("kw,code", [
    (dict(vh=0), E.KDA_ERR_WORKSPACE), (dict(knh=0), E.KDA_ERR_WORKSPACE),         # accepted up to the next check
    (dict(vh=0, vt=128, knh=0, knt=128), E.KDA_ERR_WORKSPACE), (dict(vh=0, vt=127), E.KDA_ERR_INVALID_ARG),
    (dict(knh=0, knt=0), E.KDA_ERR_INVALID_ARG), (dict(vh=0, vt=-1024), E.KDA_ERR_INVALID_ARG),
    (dict(knh=64), E.KDA_ERR_INVALID_ARG), (dict(vh=1), E.KDA_ERR_INVALID_ARG),
])
def test_expanded_shared_heads(lib, kw, code):  # noqa: F811
    """All heads may have the same keys or values; other rows may not overlap."""
    assert expanded(lib, bytes=0, **kw) == code
