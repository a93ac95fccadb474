"""Argument checks and launches shared by the ``rotary`` and ``cache`` modules."""

from __future__ import annotations

import contextlib

import torch

from . import _lib

_FLOATS = {torch.float32: _lib.GQA_F32, torch.bfloat16: _lib.GQA_BF16}
_NOTHING = contextlib.nullcontext()
# The current stream's handle; torch.cuda.current_stream builds a Stream object around it,
# 2 us of a decoding step's 20.
_current_stream = torch._C._cuda_getCurrentRawStream


def float_code(dtype) -> int:
    code = _FLOATS.get(dtype)
    if code is None:
        raise ValueError(f"dtype must be torch.float32 or torch.bfloat16, got {dtype}")
    return code


def rows(t, name, device, dtype, written=False) -> _lib.Rows:
    """The gqa_rows_t of a [B, H, L, 256] tensor.  The library checks the alignment."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != device or t.dim() != 4:
        raise ValueError(f"{name} must be a 4-d {dtype} tensor on {device}")
    B, H, L, d = t.shape
    sb, sh, sl, sd = t.stride()
    if d != 256 or sd != 1:
        raise ValueError(f"{name} must have contiguous rows of 256 columns")
    if written and ((sb == 0 and B > 1) or (sh == 0 and H > 1) or (sl == 0 and L > 1)):
        raise ValueError(f"{name} is written: its rows must not overlap")
    return _lib.Rows(t.data_ptr(), sb, sh, sl, H)


def new_like(t) -> torch.Tensor:
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def check_ints(t, shape, device, name):
    """A dense int32 tensor of this shape on the device."""
    if (not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.device != device or t.shape != shape
            or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {tuple(shape)} on {device}")
    return t


def check_positions(positions, B, L, device):
    if positions is None:
        return None
    if (not isinstance(positions, torch.Tensor) or positions.dtype != torch.int32 or positions.device != device
            or positions.shape not in ((L,), (B, L)) or (L > 1 and positions.stride(-1) != 1)):
        raise ValueError(f"positions must be an int32 tensor of shape ({L},) or ({B}, {L}) on {device}")
    return positions


def on_stream(stream):
    """Allocations made for a call on ``stream`` belong to that stream."""
    return _NOTHING if stream is None else torch.cuda.stream(stream)


def launch(name, device, stream, *args) -> None:
    """Calls the library on ``device`` and ``stream`` (default: the current one) and checks the status."""
    index = device.index
    s = _current_stream(index) if stream is None else stream.cuda_stream
    fn = getattr(_lib.load(), name)
    if torch.cuda.current_device() == index:
        rc = fn(*args, s)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, s)
    if rc:
        _lib.check(name, rc)
