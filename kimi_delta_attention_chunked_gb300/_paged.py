"""Binding of the serving-step operators (include/kda.h): block tables, cache
append, paged attention, draft verification.

As in ``_lib``, every function has the name of the C entry it calls and only
marshals arguments.  A serving step calls these for every layer, and at small
sizes the call itself is what takes the time, so the checks are written to be
cheap: no tensor is viewed or copied, and the current device is only switched
when it is another one.
"""
from __future__ import annotations

import functools

import torch

from . import _lib
from ._lib import KDA_BF16, KDA_FP32, KDA_OK, KDAError

_CODE = {torch.bfloat16: KDA_BF16, torch.float32: KDA_FP32}
_I32, _I64, _F32 = torch.int32, torch.int64, torch.float32
# the current stream's handle without a Stream object around it, where torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _call(entry, idx, stream, *args):
    """Calls C entry ``entry`` on ``stream`` with device ``idx`` current; raises on an error code."""
    fn = getattr(_lib._lib or _lib.load(), entry)
    if stream is None:
        handle = _raw_stream(idx) if _raw_stream else torch.cuda.current_stream(idx).cuda_stream
    else:
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if idx == torch.cuda.current_device():
        st = fn(*args, handle)
    else:
        with torch.cuda.device(idx):
            st = fn(*args, handle)
    if st != KDA_OK:
        raise KDAError(st, entry)


def _device(name, t):
    """Index of the CUDA device that holds t."""
    idx = t.get_device()
    if idx < 0:
        raise ValueError(f"{name} must be on a CUDA device")
    return idx


def _refuse(name, t, idx, dtype, shape):
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != idx:
        raise ValueError(f"{name} must be on cuda:{idx}")
    raise ValueError(f"{name} must be contiguous")


def _need(name, t, idx, dtype, shape):
    """Pointer of a contiguous tensor of that dtype and shape on that device."""
    if t.shape != shape or t.dtype != dtype or t.get_device() != idx or not t.is_contiguous():
        _refuse(name, t, idx, dtype, shape)
    return t.data_ptr()


def _out(name, t, like, idx, dtype, shape):
    """The caller's output tensor, checked, or a new one: (tensor, pointer)."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=like.device)
        return t, t.data_ptr()
    return t, _need(name, t, idx, dtype, shape)


def _rows(name, t, idx, dtype, shape):
    """A [tokens, heads, d] tensor whose tokens may lie further apart than heads * d
    (a slice of a fused projection): (pointer, elements between tokens)."""
    if t.shape != shape or t.dtype != dtype or t.get_device() != idx:
        _refuse(name, t, idx, dtype, shape)
    row = shape[1] * shape[2]
    if t.is_contiguous():
        return t.data_ptr(), row
    st = t.stride()
    if (st[2] != 1 and shape[2] > 1) or (st[1] != shape[2] and shape[1] > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    if shape[0] > 1 and st[0] < row:
        raise ValueError(f"{name}: tokens must not overlap")
    return t.data_ptr(), max(st[0], row)


def _code(t):
    code = _CODE.get(t.dtype)
    if code is None:
        raise TypeError(f"KDA supports bfloat16 and float32, not {t.dtype}")
    return code


def kda_build_block_tables(ctx_len, new_len, free_pages, block_table, page_size, n_tokens, cu_seqlens=None,
                           seq_len=None, slot_map=None, positions=None, n_taken=None, stream=None):
    """Lays out one serving step (include/kda.h): pages for the new tokens of every
    request, taken from ``free_pages`` [F] and written into ``block_table`` [N, blocks]
    in place, and for each of ``n_tokens`` rows of the step the cache slot and the position.
    ctx_len, new_len int32 [N].  Returns (cu_seqlens [N+1], seq_len [N], slot_map int64
    [n_tokens], positions [n_tokens], n_taken [1]); pass them in to reuse buffers."""
    if ctx_len.dim() != 1 or block_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("ctx_len and free_pages must have 1 dim, block_table 2")
    n, blocks, n_free = ctx_len.shape[0], block_table.shape[1], free_pages.shape[0]
    if new_len.shape != ctx_len.shape:
        raise ValueError(f"new_len must have shape {(n,)}, got {tuple(new_len.shape)}")
    dev = _device("ctx_len", ctx_len)
    n_tokens = int(n_tokens)
    cu_seqlens, cu_ptr = _out("cu_seqlens", cu_seqlens, ctx_len, dev, _I32, (n + 1,))
    seq_len, seq_ptr = _out("seq_len", seq_len, ctx_len, dev, _I32, (n,))
    slot_map, slot_ptr = _out("slot_map", slot_map, ctx_len, dev, _I64, (n_tokens,))
    positions, pos_ptr = _out("positions", positions, ctx_len, dev, _I32, (n_tokens,))
    n_taken, taken_ptr = _out("n_taken", n_taken, ctx_len, dev, _I32, (1,))
    _call("kda_build_block_tables", dev, stream, _need("ctx_len", ctx_len, dev, _I32, (n,)),
          _need("new_len", new_len, dev, _I32, (n,)), _need("free_pages", free_pages, dev, _I32, (n_free,)), n_free, n,
          blocks, page_size, n_tokens, _need("block_table", block_table, dev, _I32, (n, blocks)), cu_ptr, seq_ptr,
          slot_ptr, pos_ptr, taken_ptr)
    return cu_seqlens, seq_len, slot_map, positions, n_taken


def _cache_shape(name, k_cache, v_cache):
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape:
        raise ValueError(f"{name}: k_cache and v_cache must have one shape [n_pages, H_kv, page_size, d], "
                         f"got {tuple(k_cache.shape)} and {tuple(v_cache.shape)}")
    return k_cache.shape


def kda_cache_append(k, v, k_cache, v_cache, slot_map, stream=None):
    """Writes k, v [T, H_kv, d] (token stride free) to their slots of the paged caches
    [n_pages, H_kv, page_size, d], in place; slot_map int64 [T], negative slots skipped."""
    shape = _cache_shape("kda_cache_append", k_cache, v_cache)
    n_pages, heads, page, d = shape
    if k.dim() != 3:
        raise ValueError(f"k must have 3 dims, got {k.dim()}")
    rows = (k.shape[0], heads, d)
    code, dt = _code(k_cache), k_cache.dtype
    if k.shape != rows:
        raise ValueError(f"k and v must have shape {rows}, got {tuple(k.shape)} and {tuple(v.shape)}")
    if v.shape != rows:
        raise ValueError(f"k and v must have shape {rows}, got {tuple(k.shape)} and {tuple(v.shape)}")
    dev = _device("k_cache", k_cache)
    kp, ks = _rows("k", k, dev, dt, rows)
    vp, vs = _rows("v", v, dev, dt, rows)
    _call("kda_cache_append", dev, stream, kp, vp, _need("slot_map", slot_map, dev, _I64, (rows[0],)), ks, vs, rows[0],
          heads, d, page, n_pages, code, _need("k_cache", k_cache, dev, dt, shape),
          _need("v_cache", v_cache, dev, dt, shape))


@functools.lru_cache(maxsize=256)
def _workspace_size(T, heads, kv_heads, d, code):
    return int(_lib.load().kda_paged_attention_workspace_size(T, heads, kv_heads, d, code))


def kda_paged_attention_workspace_size(T: int, H_q: int, H_kv: int, d: int, dtype: torch.dtype) -> int:
    return int(_lib.load().kda_paged_attention_workspace_size(T, H_q, H_kv, d, _lib._dtype_code(dtype)))


def kda_paged_attention(q, k_cache, v_cache, block_table, cu_seqlens, seq_len, scale=None, window=0, o=None,
                        lse=None, want_lse=False, workspace=None, stream=None):
    """Attention of the new tokens q [T, H_q, d] (token stride free) over the paged caches
    [n_pages, H_kv, page_size, d] that hold their keys already (include/kda.h).
    block_table int32 [N, blocks], cu_seqlens int32 [N+1], seq_len int32 [N], all on the
    device; scale defaults to d ** -0.5; window 0 means none.  Returns o [T, H_q, d], or
    (o, lse [T, H_q] float32) where ``lse`` is passed in or ``want_lse`` is set."""
    shape = _cache_shape("kda_paged_attention", k_cache, v_cache)
    n_pages, kv_heads, page, d = shape
    if q.dim() != 3 or block_table.dim() != 2:
        raise ValueError(f"q must have 3 dims and block_table 2, got {q.dim()} and {block_table.dim()}")
    rows = q.shape
    T, heads, qd = rows
    if qd != d or heads % kv_heads != 0:
        raise ValueError(f"q {tuple(rows)} does not match caches of {kv_heads} heads of {d}")
    n, blocks = block_table.shape
    code, dt = _code(q), q.dtype
    if cu_seqlens.shape != (n + 1,) or seq_len.shape != (n,):
        raise ValueError(f"cu_seqlens and seq_len must have shapes {(n + 1,)} and {(n,)}, got "
                         f"{tuple(cu_seqlens.shape)} and {tuple(seq_len.shape)}")
    if o is not None and o.shape != rows:
        raise ValueError(f"o must have shape {tuple(rows)}, got {tuple(o.shape)}")
    if lse is not None and lse.shape != rows[:2]:
        raise ValueError(f"lse must have shape {tuple(rows[:2])}, got {tuple(lse.shape)}")
    dev = _device("q", q)
    qp, qs = _rows("q", q, dev, dt, rows)
    k_ptr, v_ptr = _need("k_cache", k_cache, dev, dt, shape), _need("v_cache", v_cache, dev, dt, shape)
    table = _need("block_table", block_table, dev, _I32, (n, blocks))
    cu, seq = _need("cu_seqlens", cu_seqlens, dev, _I32, (n + 1,)), _need("seq_len", seq_len, dev, _I32, (n,))
    o, o_ptr = _out("o", o, q, dev, dt, rows)
    lse_ptr = None
    if lse is not None or want_lse:
        lse, lse_ptr = _out("lse", lse, q, dev, _F32, rows[:2])
    if workspace is None:
        size = _workspace_size(T, heads, kv_heads, d, code)
        workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on cuda:{dev}")
    else:
        size = workspace.numel() * workspace.element_size()
    _call("kda_paged_attention", dev, stream, qp, k_ptr, v_ptr, table, cu, seq, qs, n, T, heads, kv_heads, d, page, blocks,
          n_pages, d ** -0.5 if scale is None else scale, window, code, o_ptr, lse_ptr, workspace.data_ptr(), size)
    return o if lse is None else (o, lse)


def kda_verify_draft(target, draft, draft_tokens, uniforms, draft_len=None, tokens=None, commit_len=None,
                     stream=None):
    """Decides how many drafted tokens stand and draws the next one (include/kda.h).
    target [N, K+1, V] and draft [N, K, V] probabilities of one dtype (draft None: tokens
    proposed with certainty), draft_tokens int32 [N, K], uniforms float32 [N, K+1],
    draft_len int32 [N] or None.  Returns (tokens int32 [N, K+1], commit_len int32 [N])."""
    if target.dim() != 3 or draft_tokens.dim() != 2:
        raise ValueError(f"target must have 3 dims and draft_tokens 2, got {target.dim()} and {draft_tokens.dim()}")
    n, k = draft_tokens.shape
    vocab = target.shape[2]
    if target.shape != (n, k + 1, vocab) or (draft is not None and draft.shape != (n, k, vocab)):
        raise ValueError(f"target and draft must have shapes {(n, k + 1, vocab)} and {(n, k, vocab)}, got "
                         f"{tuple(target.shape)} and {None if draft is None else tuple(draft.shape)}")
    if uniforms.shape != (n, k + 1):
        raise ValueError(f"uniforms must have shape {(n, k + 1)}, got {tuple(uniforms.shape)}")
    code, dt = _code(target), target.dtype
    dev = _device("target", target)
    ptrs = (_need("target", target, dev, dt, (n, k + 1, vocab)),
            None if draft is None else _need("draft", draft, dev, dt, (n, k, vocab)),
            _need("draft_tokens", draft_tokens, dev, _I32, (n, k)), _need("uniforms", uniforms, dev, _F32, (n, k + 1)),
            None if draft_len is None else _need("draft_len", draft_len, dev, _I32, (n,)))
    tokens, tokens_ptr = _out("tokens", tokens, target, dev, _I32, (n, k + 1))
    commit_len, commit_ptr = _out("commit_len", commit_len, target, dev, _I32, (n,))
    _call("kda_verify_draft", dev, stream, *ptrs, n, k, vocab, code, tokens_ptr, commit_ptr)
    return tokens, commit_len
