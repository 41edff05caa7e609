"""Refusals of the serving-step operators, before anything reaches a GPU: the C
ABI's own checks, and the binding's on shapes, types and strides."""
import ctypes

import pytest
import torch

import kimi_delta_attention_chunked_gb300 as kda
from kimi_delta_attention_chunked_gb300 import _lib, build

P = ctypes.c_void_p
E = _lib


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return _lib.load()


def tables(lib, **kw):
    a = dict(ctx=P(0x1000), new=P(0x2000), free=P(0x3000), n_free=4, N=2, blocks=3, page=16, n=8, table=P(0x4000),
             cu=P(0x5000), seq=P(0x6000), slot=P(0x7000), pos=P(0x8000), taken=P(0x9000))
    a.update(kw)
    return lib.kda_build_block_tables(a["ctx"], a["new"], a["free"], a["n_free"], a["N"], a["blocks"], a["page"],
                                      a["n"], a["table"], a["cu"], a["seq"], a["slot"], a["pos"], a["taken"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), E.KDA_ERR_INVALID_ARG), (dict(n_free=-1), E.KDA_ERR_INVALID_ARG),
    (dict(blocks=-1), E.KDA_ERR_INVALID_ARG), (dict(n=-1), E.KDA_ERR_INVALID_ARG),
    (dict(page=8), E.KDA_ERR_UNSUPPORTED), (dict(page=48), E.KDA_ERR_UNSUPPORTED), (dict(page=0), E.KDA_ERR_UNSUPPORTED),
    (dict(N=8193), E.KDA_ERR_UNSUPPORTED), (dict(cu=None), E.KDA_ERR_INVALID_ARG),
    (dict(taken=None), E.KDA_ERR_INVALID_ARG), (dict(ctx=None), E.KDA_ERR_INVALID_ARG),
    (dict(table=None), E.KDA_ERR_INVALID_ARG), (dict(free=None), E.KDA_ERR_INVALID_ARG),
    (dict(slot=None), E.KDA_ERR_INVALID_ARG), (dict(slot=P(0x7004)), E.KDA_ERR_INVALID_ARG),
])
def test_tables_refusals(lib, kw, code):
    assert tables(lib, **kw) == code


def append(lib, **kw):
    a = dict(k=P(0x1000), v=P(0x2000), slot=P(0x3000), ks=256, vs=256, T=4, H=2, d=128, page=16, pages=8,
             dt=E.KDA_BF16, kc=P(0x4000), vc=P(0x5000))
    a.update(kw)
    return lib.kda_cache_append(a["k"], a["v"], a["slot"], a["ks"], a["vs"], a["T"], a["H"], a["d"], a["page"],
                                a["pages"], a["dt"], a["kc"], a["vc"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), E.KDA_ERR_INVALID_ARG), (dict(H=0), E.KDA_ERR_INVALID_ARG), (dict(pages=-1), E.KDA_ERR_INVALID_ARG),
    (dict(dt=5), E.KDA_ERR_INVALID_ARG), (dict(d=96), E.KDA_ERR_UNSUPPORTED), (dict(page=20), E.KDA_ERR_UNSUPPORTED),
    (dict(ks=255), E.KDA_ERR_INVALID_ARG), (dict(vs=0), E.KDA_ERR_INVALID_ARG), (dict(k=None), E.KDA_ERR_INVALID_ARG),
    (dict(slot=None), E.KDA_ERR_INVALID_ARG), (dict(kc=P(0x4008)), E.KDA_ERR_INVALID_ARG),
    (dict(k=P(0x1001)), E.KDA_ERR_INVALID_ARG), (dict(slot=P(0x3004)), E.KDA_ERR_INVALID_ARG),
    (dict(vc=P(0x4000)), E.KDA_ERR_INVALID_ARG), (dict(kc=P(0x1000)), E.KDA_ERR_INVALID_ARG),
    (dict(T=0), E.KDA_OK), (dict(pages=0), E.KDA_OK),
])
def test_append_refusals(lib, kw, code):
    assert append(lib, **kw) == code


def attention(lib, **kw):
    a = dict(q=P(0x1000), kc=P(0x2000), vc=P(0x3000), table=P(0x4000), cu=P(0x5000), seq=P(0x6000), qs=1024, N=2, T=4,
             Hq=8, Hkv=2, d=128, page=16, blocks=4, pages=8, scale=0.1, window=0, dt=E.KDA_BF16, o=P(0x7000), lse=None,
             ws=P(0x10000), bytes=1 << 40)
    a.update(kw)
    return lib.kda_paged_attention(a["q"], a["kc"], a["vc"], a["table"], a["cu"], a["seq"], a["qs"], a["N"], a["T"],
                                   a["Hq"], a["Hkv"], a["d"], a["page"], a["blocks"], a["pages"], a["scale"],
                                   a["window"], a["dt"], a["o"], a["lse"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), E.KDA_ERR_INVALID_ARG), (dict(T=-1), E.KDA_ERR_INVALID_ARG), (dict(Hkv=3), E.KDA_ERR_INVALID_ARG),
    (dict(Hkv=0), E.KDA_ERR_INVALID_ARG), (dict(blocks=-1), E.KDA_ERR_INVALID_ARG),
    (dict(pages=-1), E.KDA_ERR_INVALID_ARG), (dict(window=-1), E.KDA_ERR_INVALID_ARG),
    (dict(dt=2), E.KDA_ERR_INVALID_ARG), (dict(d=256), E.KDA_ERR_UNSUPPORTED), (dict(page=24), E.KDA_ERR_UNSUPPORTED),
    (dict(N=8193), E.KDA_ERR_UNSUPPORTED), (dict(scale=0.0), E.KDA_ERR_INVALID_ARG),
    (dict(scale=-1.0), E.KDA_ERR_INVALID_ARG), (dict(scale=float("nan")), E.KDA_ERR_INVALID_ARG),
    (dict(scale=float("inf")), E.KDA_ERR_INVALID_ARG), (dict(qs=1023), E.KDA_ERR_INVALID_ARG),
    (dict(q=None), E.KDA_ERR_INVALID_ARG), (dict(kc=None), E.KDA_ERR_INVALID_ARG),
    (dict(table=None), E.KDA_ERR_INVALID_ARG), (dict(cu=None), E.KDA_ERR_INVALID_ARG),
    (dict(o=None), E.KDA_ERR_INVALID_ARG), (dict(o=P(0x1000)), E.KDA_ERR_INVALID_ARG),
    (dict(kc=P(0x2008)), E.KDA_ERR_INVALID_ARG), (dict(o=P(0x7008)), E.KDA_ERR_INVALID_ARG),
    (dict(q=P(0x1001)), E.KDA_ERR_INVALID_ARG), (dict(ws=None), E.KDA_ERR_WORKSPACE),
    (dict(ws=P(0x10010)), E.KDA_ERR_WORKSPACE), (dict(bytes=0), E.KDA_ERR_WORKSPACE),
    (dict(T=0), E.KDA_OK), (dict(N=0), E.KDA_OK),
])
def test_attention_refusals(lib, kw, code):
    assert attention(lib, **kw) == code


def test_attention_workspace_size(lib):
    size = lambda *a: kda.kda_paged_attention_workspace_size(*a)  # noqa: E731
    for d in (32, 64, 128):
        for dt in (torch.bfloat16, torch.float32):
            small, big = size(1, 8, 2, d, dt), size(100000, 8, 2, d, dt)
            assert 0 < small <= big < 200 << 20                    # grows with the rows of a unit, up to a limit
            assert size(200000, 8, 2, d, dt) == big
    need = size(4, 8, 2, 128, torch.bfloat16)
    assert attention(lib, bytes=need - 1) == E.KDA_ERR_WORKSPACE
    assert size(4, 8, 3, 128, torch.bfloat16) == 0 and size(4, 8, 2, 96, torch.bfloat16) == 0


def verify(lib, **kw):
    a = dict(p=P(0x1000), q=P(0x2000), t=P(0x3000), u=P(0x4000), len=None, N=2, K=4, V=100, dt=E.KDA_FP32,
             out=P(0x5000), commit=P(0x6000))
    a.update(kw)
    return lib.kda_verify_draft(a["p"], a["q"], a["t"], a["u"], a["len"], a["N"], a["K"], a["V"], a["dt"], a["out"],
                                a["commit"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), E.KDA_ERR_INVALID_ARG), (dict(K=-1), E.KDA_ERR_INVALID_ARG), (dict(V=0), E.KDA_ERR_INVALID_ARG),
    (dict(dt=9), E.KDA_ERR_INVALID_ARG), (dict(K=17), E.KDA_ERR_UNSUPPORTED), (dict(p=None), E.KDA_ERR_INVALID_ARG),
    (dict(u=None), E.KDA_ERR_INVALID_ARG), (dict(t=None), E.KDA_ERR_INVALID_ARG),
    (dict(out=None), E.KDA_ERR_INVALID_ARG), (dict(commit=None), E.KDA_ERR_INVALID_ARG),
    (dict(out=P(0x3000)), E.KDA_ERR_INVALID_ARG), (dict(N=0), E.KDA_OK),
])
def test_verify_refusals(lib, kw, code):
    assert verify(lib, **kw) == code


def z(*shape, dt=torch.float32):
    return torch.zeros(*shape, dtype=dt)


def i32(*shape):
    return z(*shape, dt=torch.int32)


def test_binding_tables():
    ok = dict(ctx_len=i32(3), new_len=i32(3), free_pages=i32(5), block_table=i32(3, 4), page_size=16, n_tokens=8)
    call = lambda **kw: kda.kda_build_block_tables(**{**ok, **kw})  # noqa: E731
    with pytest.raises(ValueError, match="CUDA device"):
        call()
    with pytest.raises(ValueError, match="dims|dim"):
        call(block_table=i32(12))
    with pytest.raises(ValueError, match="new_len"):
        call(new_len=i32(2))


def test_binding_append():
    ok = dict(k=z(5, 2, 32), v=z(5, 2, 32), k_cache=z(3, 2, 16, 32), v_cache=z(3, 2, 16, 32), slot_map=z(5, dt=torch.int64))
    call = lambda **kw: kda.kda_cache_append(**{**ok, **kw})  # noqa: E731
    with pytest.raises(ValueError, match="CUDA device"):
        call()
    with pytest.raises(ValueError, match="one shape"):
        call(v_cache=z(3, 2, 16, 64))
    with pytest.raises(ValueError, match="shape"):
        call(k=z(5, 3, 32))
    with pytest.raises(ValueError, match="shape"):
        call(v=z(4, 2, 32))
    with pytest.raises(TypeError, match="float16"):
        call(k_cache=z(3, 2, 16, 32, dt=torch.float16), v_cache=z(3, 2, 16, 32, dt=torch.float16))


def test_binding_attention():
    ok = dict(q=z(5, 4, 32), k_cache=z(3, 2, 16, 32), v_cache=z(3, 2, 16, 32), block_table=i32(2, 4), cu_seqlens=i32(3),
              seq_len=i32(2))
    call = lambda **kw: kda.kda_paged_attention(**{**ok, **kw})  # noqa: E731
    with pytest.raises(ValueError, match="CUDA device"):
        call()
    with pytest.raises(ValueError, match="does not match"):
        call(q=z(5, 3, 32))
    with pytest.raises(ValueError, match="does not match"):
        call(q=z(5, 4, 64))
    with pytest.raises(ValueError, match="cu_seqlens and seq_len"):
        call(cu_seqlens=i32(2))
    with pytest.raises(ValueError, match="cu_seqlens and seq_len"):
        call(seq_len=i32(3))
    with pytest.raises(ValueError, match="dims"):
        call(block_table=i32(8))
    with pytest.raises(ValueError, match="o must have shape"):
        call(o=z(5, 4, 31))
    with pytest.raises(ValueError, match="lse must have shape"):
        call(lse=z(5, 3))
    with pytest.raises(TypeError, match="float16"):
        call(q=z(5, 4, 32, dt=torch.float16))


def test_binding_verify():
    ok = dict(target=z(2, 4, 10), draft=z(2, 3, 10), draft_tokens=i32(2, 3), uniforms=z(2, 4))
    call = lambda **kw: kda.kda_verify_draft(**{**ok, **kw})  # noqa: E731
    with pytest.raises(ValueError, match="CUDA device"):
        call()
    with pytest.raises(ValueError, match="shapes"):
        call(target=z(2, 3, 10))
    with pytest.raises(ValueError, match="shapes"):
        call(draft=z(2, 3, 9))
    with pytest.raises(ValueError, match="uniforms"):
        call(uniforms=z(2, 3))
