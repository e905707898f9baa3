"""The norms around the gated delta rule: before the block and after it."""

from __future__ import annotations

from typing import Optional

import torch

from . import _lib
from ._host import DTYPE_CODES, _call, _fresh_like, _ptr

_ACTIVATIONS = {"sigmoid": _lib.NORM_GATE_SIGMOID, "silu": _lib.NORM_GATE_SILU,
                "swish": _lib.NORM_GATE_SILU}


def _check_weight(weight, dim, device):
    if weight is not None and (weight.dtype != torch.float32 or weight.shape != (dim,)
                               or not weight.is_contiguous() or weight.get_device() != device):
        raise ValueError(f"weight must be a contiguous float32 ({dim},) tensor on x's device, or None")


def _output(x, out):
    if out is None:
        return _fresh_like(x)
    if (out.shape != x.shape or out.dtype != x.dtype or not out.is_contiguous()
            or out.get_device() != x.get_device()):
        raise ValueError(f"out must be a contiguous {x.dtype} tensor of shape {tuple(x.shape)} on {x.device}")
    return out


def gated_rms_norm(
    x: torch.Tensor,
    gate: Optional[torch.Tensor],
    weight: Optional[torch.Tensor],
    *,
    eps: float = 1e-5,
    activation: str = "sigmoid",
    out: Optional[torch.Tensor] = None,
) -> torch.Tensor:
    """The norm after the rule, per head: x / sqrt(mean(x^2) + eps) * weight * act(gate).

    x (tokens, heads, dim) is bfloat16, float16 or float32 with a contiguous last axis, dim
    a multiple of 8 up to 512; gate has x's shape and dtype (any token and head strides), or
    is None for no gate; act is "sigmoid", or "silu" for gate * sigmoid(gate). weight (dim,)
    is float32, or None for ones. Computed in FP32 and rounded once. Queued on the current
    stream; no synchronisation.
    """
    if x.dim() != 3:
        raise ValueError("x must be (tokens, heads, dim)")
    tokens, heads, dim = x.shape
    if x.dtype not in DTYPE_CODES:
        raise ValueError(f"x must be bfloat16, float16 or float32 (got {x.dtype})")
    xs = x.stride()
    if dim > 1 and xs[2] != 1:
        raise ValueError("the last axis of x must be contiguous")
    device = x.get_device()
    if gate is None:
        code, gs = _lib.NORM_GATE_NONE, (0, 0)
    else:
        if activation not in _ACTIVATIONS:
            raise ValueError(f"unknown activation {activation!r}: use 'sigmoid' or 'silu'")
        code, gs = _ACTIVATIONS[activation], gate.stride()
        if gate.shape != x.shape or gate.dtype != x.dtype or (dim > 1 and gs[2] != 1):
            raise ValueError("gate must have x's shape and dtype and a contiguous last axis")
        if gate.get_device() != device:
            raise ValueError("gate must be on x's device")
    _check_weight(weight, dim, device)
    out = _output(x, out)
    if tokens == 0 or heads == 0:
        return out
    if not x.is_cuda:
        raise ValueError("x must be a GPU tensor")
    rc = _call(device, _lib.load().kdaconv_gated_rms_norm,
               x.data_ptr(), DTYPE_CODES[x.dtype], tokens, heads, dim, xs[0], xs[1], _ptr(gate),
               gs[0], gs[1], code, _ptr(weight), eps, out.data_ptr())
    _lib.check(rc, "gated_rms_norm")
    return out


def residual_rms_norm(
    x: torch.Tensor,
    residual: Optional[torch.Tensor],
    weight: Optional[torch.Tensor],
    *,
    eps: float = 1e-5,
    residual_scale: float = 1.0,
    out: Optional[torch.Tensor] = None,
) -> torch.Tensor:
    """The residual addition and the norm before a block::

        h = residual + residual_scale * x
        out = h / sqrt(mean(h^2) + eps) * weight

    x (tokens, hidden) is bfloat16, float16 or float32 with contiguous columns, hidden at
    most 16384. residual, of x's shape and dtype, is replaced by h rounded to that dtype; with
    None, h = residual_scale * x and is kept nowhere. out comes from the FP32 h and is rounded
    once. weight (hidden,) is float32, or None for ones. Queued on the current stream; no
    synchronisation.
    """
    if x.dim() != 2:
        raise ValueError("x must be (tokens, hidden)")
    tokens, hidden = x.shape
    if x.dtype not in DTYPE_CODES:
        raise ValueError(f"x must be bfloat16, float16 or float32 (got {x.dtype})")
    xs = x.stride()
    if hidden > 1 and xs[1] != 1:
        raise ValueError("the columns of x must be contiguous")
    device = x.get_device()
    rs = (0, 1)
    if residual is not None:
        rs = residual.stride()
        if residual.shape != x.shape or residual.dtype != x.dtype or (hidden > 1 and rs[1] != 1):
            raise ValueError("residual must have x's shape and dtype and contiguous columns")
        if residual.get_device() != device:
            raise ValueError("residual must be on x's device")
    _check_weight(weight, hidden, device)
    out = _output(x, out)
    if tokens == 0:
        return out
    if not x.is_cuda:
        raise ValueError("x must be a GPU tensor")
    rc = _call(device, _lib.load().kdaconv_residual_rms_norm,
               x.data_ptr(), DTYPE_CODES[x.dtype], tokens, hidden, xs[0], _ptr(residual), rs[0],
               residual_scale, _ptr(weight), eps, out.data_ptr())
    _lib.check(rc, "residual_rms_norm")
    return out
