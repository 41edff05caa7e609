"""The serving-step operators (include/kda.h): block tables, cache append, paged
attention, draft verification.

Every function has the name of the C entry it calls and checks its tensors
before it: shapes (ValueError), dtypes (TypeError), device and layout
(ValueError); an error code of the library raises KDAError.  The marshalling
itself is compiled (csrc/step_binding.cpp), because a serving step makes these
calls for every layer; like the library it is built by ``build.build()`` and
there is no other path.

``stream`` (a torch stream or a raw handle) names the stream of a call; without it
the call goes to the current one.  Tensors passed in must be ready there.
Tensors made for a call on another stream are memory of that stream, kept until
the current stream is done with them too; before they are used elsewhere, that
stream has to be waited for.
"""
from __future__ import annotations

import ctypes
import importlib
import os
import threading

from . import _lib

_PKG = os.path.dirname(os.path.abspath(__file__))
_lock = threading.Lock()
_binding = None


def _load():
    """The compiled binding, with the entries of libkda.so; raises if either is not built."""
    global _binding
    with _lock:
        if _binding is None:
            lib = _lib.load()
            path = os.path.join(_PKG, "_step_binding.so")
            if not os.path.exists(path):
                raise ImportError(f"KDA step binding not built: {path} is missing "
                                  "(run python -m kimi_delta_attention_chunked_gb300.build)")
            mod = importlib.import_module("._step_binding", __package__)
            entry = lambda name: ctypes.cast(getattr(lib, name), ctypes.c_void_p).value  # noqa: E731
            mod.set_entries(_lib.KDAError, entry("kda_build_block_tables"), entry("kda_cache_append"),
                            entry("kda_paged_attention_workspace_size"), entry("kda_paged_attention"),
                            entry("kda_verify_draft"), entry("kda_rotary"), entry("kda_latent_append"),
                            entry("kda_latent_attention_workspace_size"), entry("kda_latent_attention"),
                            entry("kda_expanded_attention_workspace_size"), entry("kda_expanded_attention"))
            _binding = mod
        return _binding


def kda_build_block_tables(ctx_len, new_len, free_pages, block_table, page_size, n_tokens, cu_seqlens=None,
                           seq_len=None, slot_map=None, positions=None, n_taken=None, stream=None):
    """Lays out one serving step (include/kda.h): pages for the new tokens of every
    request, taken from ``free_pages`` [F] and written into ``block_table`` [N, blocks]
    in place, and for each of ``n_tokens`` rows of the step the cache slot and the position.
    ctx_len, new_len int32 [N].  Returns (cu_seqlens [N+1], seq_len [N], slot_map int64
    [n_tokens], positions [n_tokens], n_taken [1]); pass them in to reuse buffers."""
    return (_binding or _load()).build_block_tables(ctx_len, new_len, free_pages, block_table, page_size, n_tokens,
                                                    cu_seqlens, seq_len, slot_map, positions, n_taken, stream)


def kda_cache_append(k, v, k_cache, v_cache, slot_map, stream=None):
    """Writes k, v [T, H_kv, d] (token stride free) to their slots of the paged caches
    [n_pages, H_kv, page_size, d], in place; slot_map int64 [T], negative slots skipped."""
    return (_binding or _load()).cache_append(k, v, k_cache, v_cache, slot_map, stream)


def kda_paged_attention_workspace_size(T: int, H_q: int, H_kv: int, d: int, dtype) -> int:
    return int(_lib.load().kda_paged_attention_workspace_size(T, H_q, H_kv, d, _lib._dtype_code(dtype)))


def kda_paged_attention(q, k_cache, v_cache, block_table, cu_seqlens, seq_len, scale=None, window=0, o=None,
                        lse=None, want_lse=False, workspace=None, stream=None):
    """Attention of the new tokens q [T, H_q, d] (token stride free) over the paged caches
    [n_pages, H_kv, page_size, d] that hold their keys already (include/kda.h).
    block_table int32 [N, blocks], cu_seqlens int32 [N+1], seq_len int32 [N], all on the
    device; scale defaults to d ** -0.5; window 0 means none.  Returns o [T, H_q, d], or
    (o, lse [T, H_q] float32) where ``lse`` is passed in or ``want_lse`` is set."""
    return (_binding or _load()).paged_attention(q, k_cache, v_cache, block_table, cu_seqlens, seq_len, scale, window, o,
                                                 lse, want_lse, workspace, stream)


def kda_verify_draft(target, draft, draft_tokens, uniforms, draft_len=None, tokens=None, commit_len=None,
                     stream=None):
    """Decides how many drafted tokens stand and draws the next one (include/kda.h).
    target [N, K+1, V] and draft [N, K, V] probabilities of one dtype (draft None: tokens
    proposed with certainty), draft_tokens int32 [N, K], uniforms float32 [N, K+1],
    draft_len int32 [N] or None.  Returns (tokens int32 [N, K+1], commit_len int32 [N])."""
    return (_binding or _load()).verify_draft(target, draft, draft_tokens, uniforms, draft_len, tokens, commit_len, stream)
