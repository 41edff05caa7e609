"""Refusals of the latent-attention operators, before anything reaches a GPU: the C
ABI's own checks, and the binding's on shapes, types and strides; the frequencies of
rotary positions."""
import math

import pytest
import torch

import kimi_delta_attention_chunked_gb300 as kda
from kimi_delta_attention_chunked_gb300 import _lib as E
from test_step_cpu import P, i32, lib, z  # noqa: F401

BF16 = torch.bfloat16


def rotary(lib, **kw):  # noqa: F811
    a = dict(x=P(0x1000), pos=P(0x2000), freq=P(0x3000), xt=512, xh=128, ot=512, oh=128, T=3, H=4, d=128, rot=64, inter=0,
             factor=1.0, dt=E.KDA_BF16, out=P(0x4000))
    a.update(kw)
    return lib.kda_rotary(a["x"], a["pos"], a["freq"], a["xt"], a["xh"], a["ot"], a["oh"], a["T"], a["H"], a["d"], a["rot"],
                          a["inter"], a["factor"], a["dt"], a["out"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), E.KDA_ERR_INVALID_ARG), (dict(H=0), E.KDA_ERR_INVALID_ARG), (dict(d=0, rot=0), E.KDA_ERR_INVALID_ARG),
    (dict(rot=0), E.KDA_ERR_INVALID_ARG), (dict(rot=63), E.KDA_ERR_INVALID_ARG), (dict(rot=130), E.KDA_ERR_INVALID_ARG),
    (dict(d=258, ot=2048, oh=258), E.KDA_ERR_UNSUPPORTED), (dict(H=(1 << 16) + 1), E.KDA_ERR_UNSUPPORTED),
    (dict(dt=7), E.KDA_ERR_INVALID_ARG), (dict(factor=math.nan), E.KDA_ERR_INVALID_ARG),
    (dict(factor=math.inf), E.KDA_ERR_INVALID_ARG), (dict(oh=127), E.KDA_ERR_INVALID_ARG), (dict(ot=0), E.KDA_ERR_INVALID_ARG),
    (dict(ot=500), E.KDA_ERR_INVALID_ARG),                 # neither tokens within heads nor heads within tokens
    (dict(xt=-512), E.KDA_ERR_INVALID_ARG), (dict(x=None), E.KDA_ERR_INVALID_ARG), (dict(pos=None), E.KDA_ERR_INVALID_ARG),
    (dict(freq=None), E.KDA_ERR_INVALID_ARG), (dict(out=None), E.KDA_ERR_INVALID_ARG), (dict(x=P(0x1001)), E.KDA_ERR_INVALID_ARG),
    (dict(out=P(0x4002), dt=E.KDA_FP32), E.KDA_ERR_INVALID_ARG), (dict(out=P(0x1000), ot=1024), E.KDA_ERR_INVALID_ARG),
    (dict(out=P(0x1000), oh=130, ot=1024), E.KDA_ERR_INVALID_ARG), (dict(out=P(0x2000)), E.KDA_ERR_INVALID_ARG),
    (dict(T=0), E.KDA_OK),
])
def test_rotary_refusals(lib, kw, code):  # noqa: F811
    assert rotary(lib, **kw) == code


def append(lib, **kw):  # noqa: F811
    a = dict(c=P(0x1000), r=P(0x2000), slot=P(0x3000), pos=P(0x5000), freq=P(0x6000), cs=576, rs=576, T=4, page=16, pages=8,
             inter=1, factor=1.0, dt=E.KDA_BF16, cache=P(0x4000))
    a.update(kw)
    return lib.kda_latent_append(a["c"], a["r"], a["slot"], a["pos"], a["freq"], a["cs"], a["rs"], a["T"], a["page"], a["pages"],
                                 a["inter"], a["factor"], a["dt"], a["cache"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), E.KDA_ERR_INVALID_ARG), (dict(pages=-1), E.KDA_ERR_INVALID_ARG), (dict(dt=3), E.KDA_ERR_INVALID_ARG),
    (dict(page=24), E.KDA_ERR_UNSUPPORTED), (dict(cs=511), E.KDA_ERR_INVALID_ARG), (dict(rs=63), E.KDA_ERR_INVALID_ARG),
    (dict(factor=math.nan), E.KDA_ERR_INVALID_ARG), (dict(pos=None), E.KDA_ERR_INVALID_ARG), (dict(freq=None), E.KDA_ERR_INVALID_ARG),
    (dict(c=None), E.KDA_ERR_INVALID_ARG), (dict(r=None), E.KDA_ERR_INVALID_ARG), (dict(slot=None), E.KDA_ERR_INVALID_ARG),
    (dict(cache=None), E.KDA_ERR_INVALID_ARG), (dict(cache=P(0x4008)), E.KDA_ERR_INVALID_ARG), (dict(slot=P(0x3004)), E.KDA_ERR_INVALID_ARG),
    (dict(c=P(0x1001)), E.KDA_ERR_INVALID_ARG), (dict(r=P(0x2002), dt=E.KDA_FP32), E.KDA_ERR_INVALID_ARG),
    (dict(c=P(0x4000)), E.KDA_ERR_INVALID_ARG), (dict(r=P(0x4000)), E.KDA_ERR_INVALID_ARG), (dict(T=0), E.KDA_OK), (dict(pages=0), E.KDA_OK),
])
def test_append_refusals(lib, kw, code):  # noqa: F811
    assert append(lib, **kw) == code


def absorbed(lib, **kw):  # noqa: F811
    a = dict(q=P(0x1000), cache=P(0x2000), table=P(0x4000), cu=P(0x5000), seq=P(0x6000), qs=8 * 576, N=2, T=4, H=8, page=16,
             blocks=4, pages=8, scale=0.1, dt=E.KDA_BF16, o=P(0x7000), lse=None, ws=P(0x10000), bytes=1 << 40)
    a.update(kw)
    return lib.kda_latent_attention(a["q"], a["cache"], a["table"], a["cu"], a["seq"], a["qs"], a["N"], a["T"], a["H"], a["page"],
                                    a["blocks"], a["pages"], a["scale"], a["dt"], a["o"], a["lse"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), E.KDA_ERR_INVALID_ARG), (dict(T=-1), E.KDA_ERR_INVALID_ARG), (dict(H=0), E.KDA_ERR_INVALID_ARG),
    (dict(blocks=-1), E.KDA_ERR_INVALID_ARG), (dict(pages=-1), E.KDA_ERR_INVALID_ARG), (dict(dt=2), E.KDA_ERR_INVALID_ARG),
    (dict(page=24), E.KDA_ERR_UNSUPPORTED), (dict(N=8193), E.KDA_ERR_UNSUPPORTED), (dict(H=(1 << 16) + 1), E.KDA_ERR_UNSUPPORTED),
    (dict(blocks=(2 ** 31 - 512) // 16 + 1), E.KDA_ERR_UNSUPPORTED),
    (dict(scale=0.0), E.KDA_ERR_INVALID_ARG), (dict(scale=math.nan), E.KDA_ERR_INVALID_ARG), (dict(scale=math.inf), E.KDA_ERR_INVALID_ARG),
    (dict(scale=2.0 ** 127 * 1.5), E.KDA_ERR_INVALID_ARG), (dict(qs=8 * 576 - 1), E.KDA_ERR_INVALID_ARG),
    (dict(q=None), E.KDA_ERR_INVALID_ARG), (dict(cache=None), E.KDA_ERR_INVALID_ARG), (dict(table=None), E.KDA_ERR_INVALID_ARG),
    (dict(cu=None), E.KDA_ERR_INVALID_ARG), (dict(seq=None), E.KDA_ERR_INVALID_ARG), (dict(o=None), E.KDA_ERR_INVALID_ARG),
    (dict(o=P(0x1000)), E.KDA_ERR_INVALID_ARG), (dict(o=P(0x2000)), E.KDA_ERR_INVALID_ARG), (dict(o=P(0x7010)), E.KDA_ERR_INVALID_ARG),
    (dict(cache=P(0x2008)), E.KDA_ERR_INVALID_ARG), (dict(q=P(0x1001)), E.KDA_ERR_INVALID_ARG), (dict(ws=None), E.KDA_ERR_WORKSPACE),
    (dict(ws=P(0x10010)), E.KDA_ERR_WORKSPACE), (dict(bytes=0), E.KDA_ERR_WORKSPACE), (dict(T=0), E.KDA_OK), (dict(N=0), E.KDA_OK),
])
def test_absorbed_refusals(lib, kw, code):  # noqa: F811
    assert absorbed(lib, **kw) == code


def expanded(lib, **kw):  # noqa: F811
    a = dict(q=P(0x1000), kn=P(0x2000), kr=P(0x3000), v=P(0x4000), cu=P(0x5000), cuk=P(0x6000), qs=4 * 192, knt=4 * 256, knh=256,
             krs=64, vt=4 * 256, vh=256, N=2, T=4, S=9, H=4, scale=0.1, causal=1, dt=E.KDA_BF16, o=P(0x7000), lse=None,
             ws=P(0x10000), bytes=1 << 40)
    a.update(kw)
    return lib.kda_expanded_attention(a["q"], a["kn"], a["kr"], a["v"], a["cu"], a["cuk"], a["qs"], a["knt"], a["knh"], a["krs"],
                                      a["vt"], a["vh"], a["N"], a["T"], a["S"], a["H"], a["scale"], a["causal"], a["dt"], a["o"],
                                      a["lse"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), E.KDA_ERR_INVALID_ARG), (dict(T=-1), E.KDA_ERR_INVALID_ARG), (dict(S=-1), E.KDA_ERR_INVALID_ARG),
    (dict(H=0), E.KDA_ERR_INVALID_ARG), (dict(dt=2), E.KDA_ERR_INVALID_ARG), (dict(N=8193), E.KDA_ERR_UNSUPPORTED),
    (dict(H=(1 << 16) + 1), E.KDA_ERR_UNSUPPORTED), (dict(S=2 ** 31 - 512, T=2), E.KDA_ERR_UNSUPPORTED),
    (dict(scale=-1.0), E.KDA_ERR_INVALID_ARG), (dict(scale=math.nan), E.KDA_ERR_INVALID_ARG), (dict(qs=4 * 192 - 1), E.KDA_ERR_INVALID_ARG),
    (dict(krs=63), E.KDA_ERR_INVALID_ARG), (dict(knh=127), E.KDA_ERR_INVALID_ARG), (dict(knt=800), E.KDA_ERR_INVALID_ARG),
    (dict(vt=0), E.KDA_ERR_INVALID_ARG), (dict(vh=-256), E.KDA_ERR_INVALID_ARG), (dict(q=None), E.KDA_ERR_INVALID_ARG),
    (dict(kn=None), E.KDA_ERR_INVALID_ARG), (dict(kr=None), E.KDA_ERR_INVALID_ARG), (dict(v=None), E.KDA_ERR_INVALID_ARG),
    (dict(cu=None), E.KDA_ERR_INVALID_ARG), (dict(cuk=None), E.KDA_ERR_INVALID_ARG), (dict(o=None), E.KDA_ERR_INVALID_ARG),
    (dict(o=P(0x4000)), E.KDA_ERR_INVALID_ARG), (dict(o=P(0x7010)), E.KDA_ERR_INVALID_ARG), (dict(v=P(0x4001)), E.KDA_ERR_INVALID_ARG),
    (dict(kr=P(0x3002), dt=E.KDA_FP32), E.KDA_ERR_INVALID_ARG), (dict(ws=None), E.KDA_ERR_WORKSPACE), (dict(bytes=0), E.KDA_ERR_WORKSPACE),
    (dict(ws=P(0x10080)), E.KDA_ERR_WORKSPACE), (dict(T=0), E.KDA_OK), (dict(N=0), E.KDA_OK),
])
def test_expanded_refusals(lib, kw, code):  # noqa: F811
    assert expanded(lib, **kw) == code


@pytest.mark.parametrize("size,call", [(kda.kda_latent_attention_workspace_size, absorbed),
                                       (kda.kda_expanded_attention_workspace_size, expanded)])
def test_workspace_sizes(lib, size, call):  # noqa: F811
    for H in (1, 5, 64, 65, 128):
        for dt in (BF16, torch.float32):
            small, big = size(1, H, dt), size(100000, H, dt)
            assert 0 < small <= big < 200 << 20                    # grows with the rows of a unit, up to a limit
            assert size(200000, H, dt) == big
    heads = 8 if call is absorbed else 4
    assert call(lib, bytes=size(4, heads, BF16) - 1) == E.KDA_ERR_WORKSPACE
    assert size(4, 0, BF16) == 0 and size(-1, 4, BF16) == 0


def test_binding_rotary():
    ok = dict(x=z(5, 2, 32), positions=i32(5), inv_freq=z(8))
    call = lambda **kw: kda.kda_rotary(**{**ok, **kw})  # noqa: E731
    with pytest.raises(ValueError, match="CUDA device"):
        call()
    with pytest.raises(ValueError, match="dims"):
        call(x=z(5, 32))
    with pytest.raises(ValueError, match="more pairs"):
        call(inv_freq=z(17))
    with pytest.raises(TypeError, match="float16"):
        call(x=z(5, 2, 32, dt=torch.float16))
    with pytest.raises(TypeError, match="must be a tensor"):
        call(positions=[0] * 5)
    with pytest.raises(TypeError):
        call(factor="one")


def test_binding_append():
    ok = dict(c=z(5, 512), k_rope=z(5, 64), cache=z(3, 16, 576), slot_map=z(5, dt=torch.int64))
    call = lambda **kw: kda.kda_latent_append(**{**ok, **kw})  # noqa: E731
    with pytest.raises(ValueError, match="CUDA device"):
        call()
    with pytest.raises(ValueError, match="576"):
        call(cache=z(3, 16, 512))
    with pytest.raises(ValueError, match="c must"):
        call(c=z(5, 511))
    with pytest.raises(ValueError, match="k_rope must"):
        call(k_rope=z(4, 64))
    with pytest.raises(TypeError, match="float16"):
        call(cache=z(3, 16, 576, dt=torch.float16))


def test_binding_absorbed():
    ok = dict(q=z(5, 4, 576), cache=z(3, 16, 576), block_table=i32(2, 4), cu_seqlens=i32(3), seq_len=i32(2), scale=0.1)
    call = lambda **kw: kda.kda_latent_attention(**{**ok, **kw})  # noqa: E731
    with pytest.raises(ValueError, match="CUDA device"):
        call()
    for bad in (dict(q=z(5, 4, 512)), dict(cache=z(3, 2, 16, 576)), dict(block_table=i32(8)), dict(cu_seqlens=i32(2)), dict(seq_len=i32(3))):
        with pytest.raises(ValueError, match="shape|dims"):
            call(**bad)
    with pytest.raises(TypeError, match="float16"):
        call(q=z(5, 4, 576, dt=torch.float16))
    with pytest.raises(RuntimeError, match="ambiguous"):
        call(want_lse=z(2))


def test_binding_expanded():
    ok = dict(q=z(5, 4, 192), k_nope=z(9, 4, 128), k_rope=z(9, 64), v=z(9, 4, 128), cu_seqlens=i32(3), cu_seqlens_k=i32(3))
    call = lambda **kw: kda.kda_expanded_attention(**{**ok, **kw})  # noqa: E731
    with pytest.raises(ValueError, match="CUDA device"):
        call()
    for bad in (dict(q=z(5, 4, 128)), dict(k_nope=z(9, 5, 128)), dict(k_rope=z(8, 64)), dict(v=z(9, 4, 64)), dict(cu_seqlens_k=i32(2)),
                dict(cu_seqlens=i32(0), cu_seqlens_k=i32(0))):
        with pytest.raises(ValueError, match="shape|dims|empty"):
            call(**bad)
    with pytest.raises(TypeError, match="float16"):
        call(q=z(5, 4, 192, dt=torch.float16))


def test_frequencies():
    f, factor = kda.rotary_frequencies(64, device="cpu")
    want = 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    assert factor == 1.0 and f.dtype == torch.float32 and torch.equal(f, want.float())
    f4, factor = kda.rotary_frequencies(64, scaling="linear", scale=4.0, device="cpu")
    assert factor == 1.0 and torch.equal(f4, (want / 4).float())
    ntk, _ = kda.rotary_frequencies(64, scaling="ntk", scale=8.0, device="cpu")
    assert ntk[0] == 1.0 and abs(float(ntk[-1] / f[-1]) * 8 - 1) < 1e-6             # the fastest pair stays, the slowest is slowed by 8
    y, factor = kda.rotary_frequencies(64, scaling="yarn", scale=8.0, original_length=4096, device="cpu")
    assert abs(factor - (0.1 * math.log(8.0) + 1)) < 1e-15
    turns = 4096 * want / (2 * math.pi)
    ratio = y.double() / want
    assert torch.all((ratio - 1).abs()[turns > 40] < 1e-6)                          # fast pairs keep their frequency
    assert torch.all((ratio * 8 - 1).abs()[turns < 0.8] < 1e-6)                     # slow ones are interpolated
    assert torch.all(ratio[1:] <= ratio[:-1] + 1e-6)
    for bad in (dict(dim=7), dict(dim=0), dict(dim=8, theta=1.0), dict(dim=8, scaling="cubic"), dict(dim=8, scaling="linear", scale=0.5),
                dict(dim=8, scaling="yarn", scale=2.0, original_length=0), dict(dim=2, scaling="ntk", scale=2.0)):
        with pytest.raises(ValueError):
            kda.rotary_frequencies(device="cpu", **bad)
