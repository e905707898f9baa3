"""Rotary positions: their frequencies, and the rotation of a part of every head."""

from __future__ import annotations

import math
from typing import Optional, Tuple

import torch

from . import _lib
from ._host import DTYPE_CODES, _call, _fresh_like


def rotary_frequencies(rotary_dim: int, base: float = 10000.0, *, factor: float = 1.0,
                       original_length: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0,
                       device="cuda") -> Tuple[torch.Tensor, float]:
    """Angles per position of ``rotary_dim // 2`` pairs, base ** (-2 i / rotary_dim), for
    ``rotary_embedding`` and ``latent_cache_write``, and the factor on queries and on keys.

    With ``factor`` above 1 the context is stretched that many times beyond ``original_length``
    as in YaRN (Peng et al., 2023): pairs that turn ``beta_fast`` times or more within the
    original length keep their frequency, those that turn at most ``beta_slow`` times have it
    divided by the factor, and between lies a linear ramp in the pair's number, from the first
    pair at the earliest to where a pair would turn ``beta_slow`` times, past the last one too;
    the second result is then 0.1 ln(factor) + 1, else 1. It belongs to all channels of a score:
    as ``scale`` of ``rotary_embedding`` where all of a head's channels are turned; where a part
    is, as in latent attention, its square goes into the attention's ``scale`` instead. Computed
    in FP64; the frequencies are float32.
    """
    if rotary_dim <= 0 or rotary_dim % 2:
        raise ValueError("rotary_dim must be a positive even number")
    if not base > 1 or not factor >= 1 or original_length <= 0 or not beta_fast > beta_slow > 0:
        raise ValueError("base must be above 1, factor at least 1, original_length positive and "
                         "beta_fast above beta_slow above 0")
    i = torch.arange(rotary_dim // 2, dtype=torch.float64)
    freq = base ** (-2 * i / rotary_dim)
    if factor == 1:
        return freq.float().to(device), 1.0

    def pair(turns):
        """The (fractional) number of the pair that turns so often in the original length."""
        return rotary_dim * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))

    low = max(0.0, math.floor(pair(beta_fast)))
    high = math.ceil(pair(beta_slow))
    stretched = ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
    freq = freq * (1 - stretched) + freq / factor * stretched
    return freq.float().to(device), 0.1 * math.log(factor) + 1.0


def _positions(positions, tokens, device, what="positions"):
    """Checks a vector with one index per token; returns whether it is 64 bits wide."""
    kind, size = positions.dtype, positions.shape
    if (kind is not torch.int32 and kind is not torch.int64 or len(size) != 1 or size[0] != tokens
            or not positions.is_contiguous() or positions.get_device() != device):
        raise ValueError(f"{what} must be a contiguous int32 or int64 ({tokens},) tensor on the "
                         "device of the other tensors")
    return int(kind is torch.int64)


def _frequencies(inv_freq, device):
    size = inv_freq.shape
    if (inv_freq.dtype is not torch.float32 or len(size) != 1 or not inv_freq.is_contiguous()
            or inv_freq.get_device() != device):
        raise ValueError("inv_freq must be a contiguous 1-D float32 tensor on the device of the "
                         "other tensors")
    return 2 * size[0]


def rotary_embedding(
    x: torch.Tensor,
    positions: torch.Tensor,
    inv_freq: torch.Tensor,
    *,
    offset: int = 0,
    interleaved: bool = False,
    scale: float = 1.0,
    out: Optional[torch.Tensor] = None,
) -> torch.Tensor:
    """Rotary positions on channels [offset, offset + 2 * len(inv_freq)) of every head.

    x (tokens, heads, head_dim) is bfloat16, float16 or float32 with a contiguous last axis (any
    token and head strides). Pair i, channels (2 i, 2 i + 1) counted from offset with
    ``interleaved`` and (i, i + len(inv_freq)) without, is turned by positions[t] * inv_freq[i]
    and multiplied by ``scale``. positions (tokens,) is int32 or int64; the angle is reduced in
    FP64, so far positions, up to 2^53, turn as exactly as near ones. The other channels are
    copied. ``out``, of x's shape and dtype with a contiguous last axis, may be x itself: then
    only the turned channels are read and written. Otherwise it may not overlap x. Queued on the
    current stream; no synchronisation.
    """
    size, dtype = x.shape, x.dtype
    if len(size) != 3:
        raise ValueError("x must be (tokens, heads, head_dim)")
    tokens, heads, dim = size
    if dtype not in DTYPE_CODES:
        raise ValueError(f"x must be bfloat16, float16 or float32 (got {dtype})")
    xs = x.stride()
    if dim > 1 and xs[2] != 1:
        raise ValueError("the last axis of x must be contiguous")
    device = x.get_device()
    wide = _positions(positions, tokens, device)
    rotary = _frequencies(inv_freq, device)
    if out is None:
        out = _fresh_like(x)
    elif out is not x and (out.shape != size or out.dtype is not dtype or out.get_device() != device
          or dim > 1 and out.stride()[2] != 1):
        raise ValueError(f"out must be a {dtype} tensor of shape {tuple(size)} on {x.device} "
                         "with a contiguous last axis")
    if tokens == 0 or heads == 0:
        return out
    if device < 0:
        raise ValueError("x must be a GPU tensor")
    os = xs if out is x else out.stride()
    rc = _call(device, _lib.load().kdaconv_rotary_embedding,
               x.data_ptr(), DTYPE_CODES[dtype], tokens, heads, dim, xs[0], xs[1],
               positions.data_ptr(), wide, inv_freq.data_ptr(), rotary, int(offset),
               int(interleaved), float(scale), out.data_ptr(), os[0], os[1])
    _lib.check(rc, "rotary_embedding")
    return out
