"""The speculative-decoding example: what it holds after some steps is what the
committed tokens alone give."""
import importlib.util
import os

import pytest
import torch

from _gpu import TOL_BF16, need_gpu

import kimi_delta_attention_chunked_gb300 as kda

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load():
    spec = importlib.util.spec_from_file_location("speculative_step", os.path.join(ROOT, "examples", "speculative_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("drafts", [1, 4, 7])
def test_example_state_is_that_of_the_committed_tokens(drafts):
    dev = need_gpu()
    ex = load()
    model = ex.Model(dev)
    server = ex.Server(model, n=5, drafts=drafts)
    seen = set()
    for _ in range(12):
        seen.update(server.step().tolist())
    assert len(seen) > 1                                            # some drafts stood and some did not
    ctx = server.ctx.tolist()
    assert [len(t) for t in server.text] == [c + 1 for c in ctx]
    for i, c in enumerate(ctx):
        run = torch.tensor(server.text[i][:c], device=dev)
        q, k, v, beta, la = (x[run].contiguous() for x in model.kda)
        _, S = kda.kda_prefill(q, k, v, la, beta)
        err = (server.S[i] - S[0]).abs().max() / S.abs().max()
        assert float(err) <= TOL_BF16
        pages = server.table[i, torch.arange(c, device=dev) // ex.PAGE].long()
        place = torch.arange(c, device=dev) % ex.PAGE
        assert torch.equal(server.k_cache[pages, :, place], model.k[run])
        assert torch.equal(server.v_cache[pages, :, place], model.v[run])
    assert kda.kda_get_last_device_status() == 0
