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
    size, rope_size = latents.shape, ropes.shape
    if len(size) != 3 or len(rope_size) != 3 or size[0] != rope_size[0] or size[1] != rope_size[1]:
        raise ValueError("latents must be (pages, page_size, latent_dim) and ropes (pages, page_size, "
                         "rope_dim)")
    pages, page_size, latent = size
    rope, dtype, kind = rope_size[2], ropes.dtype, latents.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise ValueError("ropes must be bfloat16 or float16")
    e4m3 = kind is not dtype
    if e4m3 and kind is not torch.float8_e4m3fn:
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
        DTYPE_CODES[dtype], e4m3)
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
    size = latent.shape
    if len(size) != 2 or size[1] != dim or rope.shape != (size[0], rope_dim):
        raise ValueError("latent must be (tokens, latent_dim) and rope (tokens, rope_dim)")
    tokens = size[0]
    if latent.dtype is not dtype or rope.dtype is not dtype:
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
    if weight is not None and (weight.dtype is not torch.float32 or weight.shape != (dim,)
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
    size = block_table.shape
    if block_table.dtype is not torch.int32 or len(size) != 2 or size[0] < seqs:
        raise ValueError("block_table must be int32 (sequences, pages per sequence)")
    ts = block_table.stride()
    if size[1] > 1 and ts[1] != 1:
        raise ValueError("the columns of block_table must be contiguous")
    if block_table.get_device() != device:
        raise ValueError("all tensors must be on the device of latents")
    return block_table.data_ptr(), ts[0], size[1]


def _loc(loc, device, what):
    size = loc.shape
    if loc.dtype is not torch.int32 or len(size) != 1 or not loc.is_contiguous():
        raise ValueError(f"{what} must be a contiguous 1-D int32 tensor")
    if loc.get_device() != device:
        raise ValueError("all tensors must be on one device")
    return size[0] - 1


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


def _queries(q_latent, q_rope, dim, rope_dim, dtype, device):
    """Checks the queries; returns (tokens, heads, latent_dim) and both tensors' strides."""
    size = q_latent.shape
    if len(size) != 3 or size[2] != dim or q_rope.shape != (size[0], size[1], rope_dim):
        raise ValueError("q_latent must be (tokens, heads, latent_dim) and q_rope (tokens, heads, rope_dim)")
    if q_latent.dtype is not dtype or q_rope.dtype is not dtype:
        raise ValueError(f"q_latent and q_rope must have the dtype of ropes, {dtype}")
    ls, rs = q_latent.stride(), q_rope.stride()
    if dim > 1 and ls[2] != 1 or rope_dim > 1 and rs[2] != 1:
        raise ValueError("the last axis of q_latent and q_rope must be contiguous")
    if q_latent.get_device() != device or q_rope.get_device() != device:
        raise ValueError("all tensors must be on the device of latents")
    return size, ls, rs


def _attend(q_latent, q_rope, latents, ropes, scales, block_table, seq_lens, query_start_loc, scale, out):
    """Checks, then kdaconv_latent_args as bytes, the output and the call's sizes."""
    cache, dim, rope_dim, dtype, device = _cache(latents, ropes, scales)
    size, ls, rs = _queries(q_latent, q_rope, dim, rope_dim, dtype, device)
    tokens, heads, _ = size
    seqs = tokens
    if query_start_loc is not None:
        seqs = max(0, _loc(query_start_loc, device, "query_start_loc"))
    lens = seq_lens.shape
    if seq_lens.dtype is not torch.int32 or len(lens) != 1 or lens[0] < seqs or (
            seqs > 1 and seq_lens.stride()[0] != 1):
        raise ValueError("seq_lens must be a contiguous 1-D int32 tensor with one entry per sequence")
    table = _table(block_table, seqs, device)
    if seq_lens.get_device() != device:
        raise ValueError("all tensors must be on the device of latents")
    if out is None:
        out = torch.empty((tokens, heads, dim), dtype=dtype, device=q_latent.device)
    elif (out.shape != size or out.dtype != dtype or not out.is_contiguous()
          or out.get_device() != device):
        raise ValueError(f"out must be a contiguous {dtype} tensor of shape {tuple(q_latent.shape)} on "
                         f"{latents.device}")
    args = cache + _lib.LATENT_ARGS.pack(
        q_latent.data_ptr(), q_rope.data_ptr(), table[0], seq_lens.data_ptr(),
        0 if query_start_loc is None else query_start_loc.data_ptr(), out.data_ptr(),
        tokens, seqs, heads, ls[0], ls[1], rs[0], rs[1], table[1], table[2], float(scale))
    return args, out, device, (tokens, seqs, heads, dim)


def _run(name, args, out, device, sizes):
    if 0 in sizes:
        return out
    if device < 0:
        raise ValueError("latents must be a GPU tensor")
    lib = _lib.load()
    # Memory of the current stream: the allocator hands it out again only to work that is
    # queued behind this call.
    need = lib.kdaconv_latent_attention_workspace(*sizes)
    scratch = torch.empty(need, dtype=torch.uint8, device=out.device)
    rc = _call(device, getattr(lib, "kdaconv_" + name), args, scratch.data_ptr(), need)
    _lib.check(rc, name)
    return out


def latent_attention_fn(
    q_latent: torch.Tensor,
    q_rope: torch.Tensor,
    latents: torch.Tensor,
    ropes: torch.Tensor,
    scales: Optional[torch.Tensor],
    block_table: torch.Tensor,
    seq_lens: torch.Tensor,
    query_start_loc: torch.Tensor,
    *,
    scale: float,
    out: Optional[torch.Tensor] = None,
) -> torch.Tensor:
    """Attention of packed new tokens over the paged latent cache, in the absorbed form.

    For every head of token i of the n new tokens of a sequence, over the sequence's tokens t <
    seq_lens - n + i + 1 (the new ones are in the cache already)::

        s_t = scale * (q_latent . latent_t + q_rope . rope_t)
        out = sum_t softmax(s)_t latent_t

    q_latent (tokens, heads, latent_dim) is the query times the latents' up-projection for the
    keys, q_rope (tokens, heads, rope_dim) its turned part, both of ropes' dtype with a contiguous
    last axis (any token and head strides); the result (tokens, heads, latent_dim) is still to be
    multiplied by the up-projection for the values. ``scale`` is that of the unabsorbed heads,
    (key channels + rope_dim) ** -0.5.

    latents, ropes and scales are the cache of ``latent_cache_write``, block_table (sequences,
    pages per sequence) int32 its pages, seq_lens (sequences,) int32 the tokens of each sequence
    in it, the new ones included, and query_start_loc (sequences + 1,) int32 the rows of each. A
    token whose page is outside the cache is not there; a row that sees no token, or only scores
    of -inf, is zero; rows no sequence owns are left unwritten; a latent that is not finite reaches
    no row that does not see it. Scores, softmax and sums are FP32, the weights rounded to the
    dtype for the second product, the result rounded once. Takes up to 67 MB of scratch memory
    from torch's allocator. Queued on the current stream; no synchronisation.
    """
    return _run("latent_attention", *_attend(q_latent, q_rope, latents, ropes, scales, block_table,
                                             seq_lens, query_start_loc, scale, out))


def latent_attention_update(
    q_latent: torch.Tensor,
    q_rope: torch.Tensor,
    latents: torch.Tensor,
    ropes: torch.Tensor,
    scales: Optional[torch.Tensor],
    block_table: torch.Tensor,
    seq_lens: torch.Tensor,
    *,
    scale: float,
    out: Optional[torch.Tensor] = None,
) -> torch.Tensor:
    """Decode step of ``latent_attention_fn``: row b of q_latent and q_rope is the one new token
    of sequence b, which sees all seq_lens[b] tokens. Arguments and result as there."""
    return _run("latent_attention_update", *_attend(q_latent, q_rope, latents, ropes, scales,
                                                    block_table, seq_lens, None, scale, out))


def latent_attention_supported(q_latent: torch.Tensor, q_rope: torch.Tensor, latents: torch.Tensor,
                               ropes: torch.Tensor, scales: Optional[torch.Tensor] = None) -> bool:
    """Whether latent_attention_fn and latent_attention_update serve these tensors."""
    try:
        cache, dim, rope_dim, dtype, device = _cache(latents, ropes, scales)
        (tokens, heads, _), ls, rs = _queries(q_latent, q_rope, dim, rope_dim, dtype, device)
        lib = _lib.load()
    except (ValueError, _lib.LibraryMissing):
        return False
    # What a call has beside these is aligned: any such address will do.
    args = cache + _lib.LATENT_ARGS.pack(q_latent.data_ptr(), q_rope.data_ptr(), 256, 256, 0, 256, tokens, tokens, heads,
                                         ls[0], ls[1], rs[0], rs[1], 1, 1, 1.0)
    return device >= 0 and lib.kdaconv_latent_attention_validate(args, 1, 256, 1 << 62) == _lib.OK
