"""Host-side helpers the bindings share: formats, the current stream and device."""

from __future__ import annotations

from typing import Optional

import torch

from . import _lib

# Tensor formats the library takes, with their interface codes.
DTYPE_CODES = {torch.bfloat16: _lib.BF16, torch.float16: _lib.F16, torch.float32: _lib.F32}

#: Default null block id. The page names the default (NULL_BLOCK_ID) without
#: printing its value; 0, the block the paged cache reserves as its null block,
#: is taken here. Pass the id explicitly (or None) to be independent of this.
NULL_BLOCK_ID = 0

# The current stream's raw handle: torch's direct query where it has one (0.1 us against
# about 2 us for building a Stream object per call), else the public route.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# The current device, likewise by the direct query where torch has one (a plain call,
# without the initialisation checks of torch.cuda.current_device()).
_get_device = getattr(torch._C, "_cuda_getDevice", None)


def _current_device() -> int:
    return _get_device() if _get_device is not None else torch.cuda.current_device()


def _stream_handle(device: torch.device) -> int:
    if _raw_stream is not None:
        idx = device.index if device.index is not None else _current_device()
        return _raw_stream(idx)
    return torch.cuda.current_stream(device).cuda_stream


class _NoGuard:
    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


_NO_GUARD = _NoGuard()


def _on(device: torch.device):
    """The device context for a call on `device`: none when it is already current (the
    context manager costs more than the launch's own host work)."""
    if device.index is None or device.index == _current_device():
        return _NO_GUARD
    return torch.cuda.device(device)


def _stream_of(index: int) -> int:
    """The raw current stream of device `index`."""
    return _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(index).cuda_stream


def _call(index: int, function, *args) -> int:
    """function(*args, current stream of device `index`) with that device current."""
    if index == _current_device():
        return function(*args, _stream_of(index))
    with torch.cuda.device(index):
        return function(*args, _stream_of(index))


def _fresh_like(t: torch.Tensor) -> torch.Tensor:
    """A contiguous tensor of t's shape, dtype and device (half the host time of torch.empty)."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()
