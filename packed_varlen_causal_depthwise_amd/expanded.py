"""Attention of packed sequences with keys and values expanded for every head."""

from __future__ import annotations

from typing import Optional

import torch

from . import _lib
from ._host import DTYPE_CODES, _call, _ptr
from .latent import _loc


def _inputs(q, k, k_rope, v):
    """Checks them; returns kdaconv_expanded_args' sizes and strides."""
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3 or k.shape[:2] != v.shape[:2] or q.shape[1] != k.shape[1]:
        raise ValueError("q must be (tokens, heads, key_dim + rope_dim), k (keys, heads, key_dim) and "
                         "v (keys, heads, value_dim)")
    tokens, heads, width = q.shape
    keys, _, key_dim = k.shape
    value_dim, dtype = v.shape[2], q.dtype
    rope_dim = 0 if k_rope is None else k_rope.shape[-1]
    if k_rope is not None and k_rope.shape != (keys, rope_dim):
        raise ValueError("k_rope must be (keys, rope_dim), or None")
    if width != key_dim + rope_dim:
        raise ValueError(f"q has {width} channels, k and k_rope have {key_dim} and {rope_dim}")
    if dtype not in (torch.bfloat16, torch.float16) or k.dtype != dtype or v.dtype != dtype or (
            k_rope is not None and k_rope.dtype != dtype):
        raise ValueError("q, k, k_rope and v must share one dtype: bfloat16 or float16")
    qs, ks, vs = q.stride(), k.stride(), v.stride()
    rs = (0, 1) if k_rope is None else k_rope.stride()
    if (width > 1 and qs[2] != 1 or key_dim > 1 and ks[2] != 1 or value_dim > 1 and vs[2] != 1
            or rope_dim > 1 and rs[1] != 1):
        raise ValueError("the last axis of q, k, k_rope and v must be contiguous")
    device = q.get_device()
    if k.get_device() != device or v.get_device() != device or (
            k_rope is not None and k_rope.get_device() != device):
        raise ValueError("all tensors must be on the device of q")
    return ((tokens, keys, heads, key_dim, rope_dim, value_dim),
            (qs[0], qs[1], ks[0], ks[1], rs[0], vs[0], vs[1]))


def _pack(q, k, k_rope, v, loc, kv_loc, out, seqs, sizes, strides, scale, causal):
    """kdaconv_expanded_args as bytes; loc, kv_loc and out are addresses."""
    tokens, keys, heads, key_dim, rope_dim, value_dim = sizes
    return _lib.EXPANDED_ARGS.pack(
        q.data_ptr(), k.data_ptr(), 0 if k_rope is None else k_rope.data_ptr(), v.data_ptr(), loc, kv_loc, out,
        tokens, keys, max(0, seqs), heads, key_dim, rope_dim, value_dim, *strides,
        (key_dim + rope_dim or 1) ** -0.5 if scale is None else float(scale), DTYPE_CODES[q.dtype], int(causal))


def _expand(q, k, k_rope, v, query_start_loc, kv_start_loc, scale, causal, out):
    """Checks, then kdaconv_expanded_args as bytes, the output and the call's sizes."""
    sizes, strides = _inputs(q, k, k_rope, v)
    tokens, keys, heads, _, _, value_dim = sizes
    dtype, device = q.dtype, q.get_device()
    seqs = _loc(query_start_loc, device, "query_start_loc")
    if kv_start_loc is None:
        kv_start_loc = query_start_loc
    elif _loc(kv_start_loc, device, "kv_start_loc") != seqs:
        raise ValueError("kv_start_loc must have as many entries as query_start_loc")
    shape = (tokens, heads, value_dim)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=q.device)
    elif out.shape != shape or out.dtype != dtype or not out.is_contiguous() or out.get_device() != device:
        raise ValueError(f"out must be a contiguous {dtype} tensor of shape {shape} on {q.device}")
    args = _pack(q, k, k_rope, v, query_start_loc.data_ptr(), kv_start_loc.data_ptr(), out.data_ptr(), seqs, sizes,
                 strides, scale, causal)
    return args, out, (tokens, keys, seqs, heads, value_dim)


def expanded_attention_fn(
    q: torch.Tensor,
    k: torch.Tensor,
    k_rope: Optional[torch.Tensor],
    v: torch.Tensor,
    query_start_loc: torch.Tensor,
    kv_start_loc: Optional[torch.Tensor] = None,
    *,
    scale: Optional[float] = None,
    causal: bool = True,
    out: Optional[torch.Tensor] = None,
) -> torch.Tensor:
    """Attention of packed sequences in the expanded form of latent attention (prefill).

    Queries rows query_start_loc[s] .. of sequence s over its keys, rows kv_start_loc[s] .. (None:
    the same rows as the queries). With ``causal`` query i of n sees the first m - n + i + 1 of m
    keys, so that queries are the sequence's last tokens; without, all of them::

        s_t = scale * (q[:key_dim] . k_t + q[key_dim:] . k_rope_t)
        out = sum_t softmax(s)_t v_t

    q (tokens, heads, key_dim + rope_dim), k (keys, heads, key_dim) and v (keys, heads, value_dim)
    are bfloat16 or float16 with a contiguous last axis and any token and head strides (a token of
    k, k_rope and v below 2^23 elements from the next): k and v may be slices of one
    up-projection's rows. k_rope (keys, rope_dim), a slice of ``latent_cache_read``'s rows say, is
    the part of the keys that all heads share, or None. scale defaults to
    (key_dim + rope_dim) ** -0.5; 0 is allowed. key_dim and value_dim are multiples of 8 up to
    128, rope_dim up to 64; k, k_rope and v lie at multiples of 16 bytes, row for row and head for
    head.

    A row that sees no key, or only scores of -inf, is zero, rows no sequence owns are left
    unwritten, and a value that is not finite reaches no row that does not see it (that channel of
    those that do is NaN or infinite). Scores, softmax and sums are FP32, the weights rounded to
    the dtype for the second product, the result (tokens, heads, value_dim) once. Few rows over
    many keys take up to 35 MB of scratch memory from torch's allocator. Queued on the current
    stream; no synchronisation.
    """
    args, out, sizes = _expand(q, k, k_rope, v, query_start_loc, kv_start_loc, scale, causal, out)
    tokens, _, seqs, heads, _ = sizes
    if tokens == 0 or seqs <= 0 or heads == 0:
        return out
    device = q.get_device()
    if device < 0:
        raise ValueError("q must be a GPU tensor")
    lib = _lib.load()
    need, scratch = lib.kdaconv_expanded_attention_workspace(*sizes), None
    if need:  # memory of the current stream, as the attention over the cache takes it
        scratch = torch.empty(need, dtype=torch.uint8, device=out.device)
    rc = _call(device, lib.kdaconv_expanded_attention, args, _ptr(scratch), need)
    _lib.check(rc, "expanded_attention_fn")
    return out


def expanded_attention_supported(q: torch.Tensor, k: torch.Tensor, k_rope: Optional[torch.Tensor],
                                 v: torch.Tensor) -> bool:
    """Whether expanded_attention_fn serves these tensors."""
    try:
        sizes, strides = _inputs(q, k, k_rope, v)
        lib = _lib.load()
    except (ValueError, _lib.LibraryMissing):
        return False
    # What a call has beside these is aligned: any such address will do.
    args = _pack(q, k, k_rope, v, 256, 256, 256, 1, sizes, strides, 1.0, True)
    return q.get_device() >= 0 and lib.kdaconv_expanded_attention_validate(args, 256, 1 << 62) == _lib.OK
