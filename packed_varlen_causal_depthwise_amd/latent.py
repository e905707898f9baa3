"""Latent attention: its paged cache, and attention over it."""

from __future__ import annotations

from typing import Optional

import torch

from . import _lib
from ._host import DTYPE_CODES, _call, _ptr
from .rotary import _frequencies, _positions

#: Channels of a latent that share one scale in the 8-bit cache.
SCALE_BLOCK = 32


def _cache(latents, ropes, scales):
    """Checks a cache's tensors; returns kdaconv_latent_cache as bytes and its sizes."""
    if latents.dim() != 3 or ropes.dim() != 3 or latents.shape[:2] != ropes.shape[:2]:
        raise ValueError("latents must be (pages, page_size, latent_dim) and ropes (pages, page_size, "
                         "rope_dim)")
    pages, page_size, latent = latents.shape
    rope, dtype = ropes.shape[2], ropes.dtype
    if dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("ropes must be bfloat16 or float16")
    e4m3 = latents.dtype == torch.float8_e4m3fn
    if not e4m3 and latents.dtype != dtype:
        raise ValueError("latents must have the dtype of ropes, or float8_e4m3fn")
    ls, rs, ss = latents.stride(), ropes.stride(), (0, 0)
    if latent > 1 and ls[2] != 1 or rope > 1 and rs[2] != 1:
        raise ValueError("the last axis of latents and ropes must be contiguous")
    device = latents.get_device()
    if e4m3:
        blocks = latent // SCALE_BLOCK
        if scales is None or scales.dtype != torch.uint8 or scales.shape != (pages, page_size, blocks):
            raise ValueError("float8_e4m3fn latents need uint8 scales (pages, page_size, latent_dim // "
                             f"{SCALE_BLOCK}), exponents plus 127")
        ss = scales.stride()
        if blocks > 1 and ss[2] != 1:
            raise ValueError("the last axis of scales must be contiguous")
    elif scales is not None:
        raise ValueError("scales belong to float8_e4m3fn latents")
    if ropes.get_device() != device or scales is not None and scales.get_device() != device:
        raise ValueError("all tensors must be on the device of latents")
    packed = _lib.LATENT_CACHE.pack(
        latents.data_ptr(), ropes.data_ptr(), 0 if scales is None else scales.data_ptr(),
        pages, page_size, latent, rope, ls[0], ls[1], rs[0], rs[1], ss[0], ss[1],
        DTYPE_CODES[dtype], int(e4m3))
    return packed, latent, rope, dtype, device


def latent_cache_write(
    latent: torch.Tensor,
    rope: torch.Tensor,
    latents: torch.Tensor,
    ropes: torch.Tensor,
    scales: Optional[torch.Tensor],
    slots: torch.Tensor,
    *,
    weight: Optional[torch.Tensor] = None,
    eps: Optional[float] = None,
    positions: Optional[torch.Tensor] = None,
    inv_freq: Optional[torch.Tensor] = None,
    interleaved: bool = False,
    rope_scale: float = 1.0,
) -> None:
    """Writes new tokens into the paged cache of latent attention, in place.

    latent (tokens, latent_dim) and rope (tokens, rope_dim), bfloat16 or float16 with contiguous
    columns, are what the down-projection gives: one latent and one vector to rotate a token, for
    all heads. With ``eps`` the latent is normed first, latent / sqrt(mean(latent^2) + eps) *
    weight (weight float32 (latent_dim,), None for ones); with ``inv_freq`` (rope_dim / 2,) rope
    is turned by ``positions`` as in ``rotary_embedding`` (``rope_scale`` is its ``scale``).

    latents (pages, page_size, latent_dim) and ropes (pages, page_size, rope_dim) have that dtype
    and a contiguous last axis; they may be slices of one tensor. Or latents is float8_e4m3fn, with
    scales (pages, page_size, latent_dim // 32) uint8: each block of 32 channels is held as 8-bit
    values times 2^(scale - 127), the smallest power of two of at least 2^-100 with which they
    stay at most 448; infinities and NaN become NaN. Else scales is None. Token t goes to place
    slots[t] % page_size of page slots[t] // page_size; slots (tokens,) is int32 or int64, and a
    token whose slot is outside the cache (-1, say) is left out. Slots in the cache are distinct.

    latent_dim is a multiple of 8 (32 for 8 bits) up to 512, rope_dim one of 8 up to 64, 0 included;
    rows of latents and ropes lie at multiples of 16 bytes. Queued on the current stream; no
    synchronisation.
    """
    cache, dim, rope_dim, dtype, device = _cache(latents, ropes, scales)
    if latent.dim() != 2 or latent.shape[1] != dim or rope.shape != (latent.shape[0], rope_dim):
        raise ValueError("latent must be (tokens, latent_dim) and rope (tokens, rope_dim)")
    tokens = latent.shape[0]
    if latent.dtype != dtype or rope.dtype != dtype:
        raise ValueError(f"latent and rope must have the dtype of ropes, {dtype}")
    xs, rs = latent.stride(), rope.stride()
    if dim > 1 and xs[1] != 1 or rope_dim > 1 and rs[1] != 1:
        raise ValueError("the columns of latent and rope must be contiguous")
    if latent.get_device() != device or rope.get_device() != device:
        raise ValueError("all tensors must be on the device of latents")
    wide = _positions(slots, tokens, device, "slots")
    if eps is None:
        if weight is not None:
            raise ValueError("weight belongs to the norm: give eps")
    elif not eps >= 0:
        raise ValueError("eps must not be negative")
    if weight is not None and (weight.dtype != torch.float32 or weight.shape != (dim,)
                               or not weight.is_contiguous() or weight.get_device() != device):
        raise ValueError(f"weight must be a contiguous float32 ({dim},) tensor on the device of latents")
    far = 0
    if inv_freq is not None:
        if _frequencies(inv_freq, device) != rope_dim:
            raise ValueError("inv_freq must have rope_dim / 2 entries")
        if positions is None:
            raise ValueError("inv_freq needs positions")
        far = _positions(positions, tokens, device)
    if tokens == 0:
        return
    if device < 0:
        raise ValueError("latents must be a GPU tensor")
    rc = _call(device, _lib.load().kdaconv_latent_cache_write,
               cache, latent.data_ptr(), xs[0], rope.data_ptr(), rs[0], tokens, slots.data_ptr(), wide,
               _ptr(weight), -1.0 if eps is None else float(eps),
               None if inv_freq is None else positions.data_ptr(), far,
               _ptr(inv_freq) if rope_dim else None, int(interleaved), float(rope_scale))
    _lib.check(rc, "latent_cache_write")


def _table(block_table, seqs, device):
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] < seqs:
        raise ValueError("block_table must be int32 (sequences, pages per sequence)")
    ts = block_table.stride()
    if block_table.shape[1] > 1 and ts[1] != 1:
        raise ValueError("the columns of block_table must be contiguous")
    if block_table.get_device() != device:
        raise ValueError("all tensors must be on the device of latents")
    return block_table.data_ptr(), ts[0], block_table.shape[1]


def _loc(loc, device, what):
    if loc.dtype != torch.int32 or loc.dim() != 1 or not loc.is_contiguous():
        raise ValueError(f"{what} must be a contiguous 1-D int32 tensor")
    if loc.get_device() != device:
        raise ValueError("all tensors must be on one device")
    return loc.shape[0] - 1


def latent_cache_read(
    latents: torch.Tensor,
    ropes: torch.Tensor,
    scales: Optional[torch.Tensor],
    block_table: torch.Tensor,
    kv_start_loc: torch.Tensor,
    num_tokens: int,
    *,
    out: Optional[torch.Tensor] = None,
) -> torch.Tensor:
    """Packed sequences out of the paged cache: (num_tokens, latent_dim + rope_dim) in ropes'
    dtype, latents in the first columns (8-bit ones times their scales, rounded once).

    Token i of sequence s, row kv_start_loc[s] + i of the result, lies in page
    block_table[s, i // page_size]. block_table (sequences, pages per sequence) and kv_start_loc
    (sequences + 1,) are int32. Rows that no sequence owns are left unwritten; tokens on pages
    outside the cache read as zeros. The cache's tensors are those of ``latent_cache_write``;
    ``out`` is contiguous and aligned to 16 bytes. Queued on the current stream; no
    synchronisation.
    """
    cache, dim, rope_dim, dtype, device = _cache(latents, ropes, scales)
    seqs = _loc(kv_start_loc, device, "kv_start_loc")
    shape = (int(num_tokens), dim + rope_dim)
    table = _table(block_table, seqs, device)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=latents.device)
    elif out.shape != shape or out.dtype != dtype or not out.is_contiguous() or out.get_device() != device:
        raise ValueError(f"out must be a contiguous {dtype} tensor of shape {shape} on {latents.device}")
    if shape[0] == 0 or seqs <= 0:
        return out
    if device < 0:
        raise ValueError("latents must be a GPU tensor")
    rc = _call(device, _lib.load().kdaconv_latent_cache_read, cache, *table,
               kv_start_loc.data_ptr(), seqs, shape[0], out.data_ptr())
    _lib.check(rc, "latent_cache_read")
    return out
