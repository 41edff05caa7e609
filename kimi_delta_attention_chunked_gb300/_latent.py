"""Latent attention (include/kda.h): rotary positions, the paged latent cache,
absorbed and expanded attention.

Functions that carry the name of a C entry check their tensors before they call
it, as the other step operators do (``_paged``), through the same compiled
binding; ``stream`` means the same here.
"""
from __future__ import annotations

import math

from . import _lib, _paged


def rotary_frequencies(dim: int, theta: float = 10000.0, scaling=None, scale: float = 1.0, original_length: int = 4096,
                       beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda"):
    """Frequencies of ``dim`` / 2 channel pairs in radians a position, and the factor that goes with them.

    Unscaled, pair i has theta ** (-2 i / dim).  For contexts ``scale`` times as long as the
    ``original_length`` that a model was trained on:

    * "linear": every frequency divided by ``scale`` (position interpolation);
    * "ntk": theta raised so that the slowest pair is slowed by ``scale``, the fastest not at all;
    * "yarn": pairs that turn more than ``beta_fast`` times over the original length keep their
      frequency, those that turn less than ``beta_slow`` times are divided by ``scale``, with a ramp
      between; the factor is 0.1 ln(scale) + 1 (YaRN, Peng et al. 2023, section 3).

    Returns (inv_freq float32 [dim / 2] on ``device``, factor); formed in 64 bits, rounded once."""
    import torch
    if dim < 2 or dim % 2:
        raise ValueError(f"dim must be even and positive, got {dim}")
    if not (theta > 1.0 and math.isfinite(theta)):
        raise ValueError(f"theta must be above 1, got {theta}")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f'scaling must be None, "linear", "ntk" or "yarn", got {scaling!r}')
    if not (scale >= 1.0 and math.isfinite(scale)):
        raise ValueError(f"scale must be at least 1, got {scale}")
    i = torch.arange(0, dim, 2, dtype=torch.float64)
    factor = 1.0
    if scaling == "ntk":
        if dim < 4:
            raise ValueError("ntk scaling needs two pairs or more")
        theta = theta * scale ** (dim / (dim - 2))
    freq = theta ** (-i / dim)
    if scaling == "linear":
        freq = freq / scale
    elif scaling == "yarn":
        if original_length <= 0 or not beta_fast > beta_slow > 0:
            raise ValueError("yarn scaling needs a positive original_length and beta_fast > beta_slow > 0")
        # the (fractional) pair that turns `turns` times over the original length
        pair = lambda turns: dim * math.log(original_length / (2 * math.pi * turns)) / (2 * math.log(theta))  # noqa: E731
        low, high = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), dim - 1)
        ramp = ((i / 2 - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)
        freq = freq * (1 - ramp) + freq / scale * ramp
        factor = 0.1 * math.log(scale) + 1.0
    return freq.float().to(device), factor


def kda_rotary(x, positions, inv_freq, factor=1.0, interleaved=False, out=None, stream=None):
    """Turns the first 2 * len(inv_freq) channels of every head of x [T, H, d] by its token's position
    (include/kda.h) and copies the others.  positions int32 [T], inv_freq float32, both on the device.
    x and out may be views (any token and head strides, the channels contiguous); out None: a new
    tensor; out=x: in place.  Returns out."""
    return (_paged._binding or _paged._load()).rotary(x, positions, inv_freq, factor, interleaved, out, stream)


def kda_latent_append(c, k_rope, cache, slot_map, positions=None, inv_freq=None, factor=1.0, interleaved=False, stream=None):
    """Writes latents c [T, 512] and key parts k_rope [T, 64] (token strides free) to their slots of the
    paged latent cache [n_pages, page_size, 576], in place; with positions int32 [T] and inv_freq
    float32 [32] the key part is turned on the way.  slot_map int64 [T], negative slots skipped."""
    return (_paged._binding or _paged._load()).latent_append(c, k_rope, cache, slot_map, positions, inv_freq, factor,
                                                             interleaved, stream)


def kda_latent_attention_workspace_size(T: int, H: int, dtype) -> int:
    return int(_lib.load().kda_latent_attention_workspace_size(T, H, _lib._dtype_code(dtype)))


def kda_latent_attention(q, cache, block_table, cu_seqlens, seq_len, scale, o=None, lse=None, want_lse=False, workspace=None,
                         stream=None):
    """Absorbed attention of the new tokens q [T, H, 576] (token stride free) over the paged latent cache
    [n_pages, page_size, 576] that holds their rows already (include/kda.h).  block_table int32
    [N, blocks], cu_seqlens int32 [N+1], seq_len int32 [N], all on the device; scale is the expanded
    head's.  Returns o [T, H, 512], or (o, lse [T, H] float32) where ``lse`` is passed in or ``want_lse``
    is set."""
    return (_paged._binding or _paged._load()).latent_attention(q, cache, block_table, cu_seqlens, seq_len, scale, o, lse,
                                                                want_lse, workspace, stream)


def kda_expanded_attention_workspace_size(T: int, H: int, dtype) -> int:
    return int(_lib.load().kda_expanded_attention_workspace_size(T, H, _lib._dtype_code(dtype)))


def kda_expanded_attention(q, k_nope, k_rope, v, cu_seqlens, cu_seqlens_k, scale=None, causal=True, o=None, lse=None,
                           want_lse=False, workspace=None, stream=None):
    """Expanded attention of q [T, H, 192] over packed keys and values (include/kda.h): k_nope [S, H, 128],
    k_rope [S, 64] shared by the heads, v [S, H, 128], views with free token and head strides whose rows
    do not overlap (expanded over the heads: one row for all of them, on CUDA cores); cu_seqlens and cu_seqlens_k int32 [N+1] on the device.  scale defaults to 192 ** -0.5.  Returns
    o [T, H, 128], or (o, lse [T, H] float32) where ``lse`` is passed in or ``want_lse`` is set."""
    return (_paged._binding or _paged._load()).expanded_attention(q, k_nope, k_rope, v, cu_seqlens, cu_seqlens_k, scale, causal,
                                                                  o, lse, want_lse, workspace, stream)
