"""Rotary positions for queries and keys (``gqa_attn_rope``).

Pair i of the first ``rot`` columns of a row at position p turns by the angle p f_i:

    y1 = m (x1 cos a - x2 sin a),    y2 = m (x2 cos a + x1 sin a),    a = p f_i

with pairs (i, i + rot / 2) (``layout="half"``) or (2i, 2i + 1) (``"interleaved"``); the
other columns stay.  A ``Table`` holds the frequencies: plain, scaled for long contexts,
or the caller's own.

    table = rotary.Table(rot=128, scaling="yarn", factor=8.0, original_length=8192)
    q, k = rotary.rotate(q, k, table)                              # positions 0 .. L - 1
    q, k = rotary.rotate(q, k, table, positions=ids)               # any int32 positions, [L] or [B, L]
    q, k = rotary.rotate_autograd(q, k, table)                     # differentiable

q, k: [B, H, L, 256], fp32 or bf16, rows contiguous, the other dimensions in any strides
of whole 16 bytes (a projection's [B, L, H, 256] viewed as [B, H, L, 256] needs no copy).
"""

from __future__ import annotations

import ctypes

import torch

from . import _device, _lib
from ._views import check_positions, float_code, launch, new_like, on_stream, rows

LAYOUTS = {"half": 0, "interleaved": 1}
SCALINGS = {None: 0, "none": 0, "linear": 1, "ntk": 2, "yarn": 3}


class Table:
    """Frequencies of a rotation and their device copies.

    ``rot``: rotated columns, a multiple of 16 up to 256.  ``scaling``: ``None``,
    ``"linear"`` (positions divided by ``factor``), ``"ntk"`` (``base`` raised so that the
    slowest pair slows by ``factor``) or ``"yarn"`` (pairs that turn fewer than
    ``beta_slow`` times over ``original_length`` slow by ``factor``, those above
    ``beta_fast`` do not, and the magnitude is 0.1 ln(factor) + 1; between the two the
    ramp is linear in the turns, as in the paper: for a checkpoint whose loader ramps in the pair's
    index, between bounds rounded to whole pairs, give its frequencies).  ``inv_freq`` (a
    sequence of rot / 2 numbers, with ``magnitude``) replaces all of that by the caller's
    own.  The words the kernels read are copied to ``device`` here, and to another device
    by its first call there: make that call, or ``table.on(device)``, before a capture."""

    def __init__(self, rot=256, *, base=10000.0, layout="half", scaling=None, factor=1.0, original_length=0,
                 beta_fast=32.0, beta_slow=1.0, inv_freq=None, magnitude=None, device=None):
        if layout not in LAYOUTS:
            raise ValueError(f"layout must be one of {tuple(LAYOUTS)}, got {layout!r}")
        if scaling not in SCALINGS:
            raise ValueError(f"scaling must be one of {tuple(SCALINGS)}, got {scaling!r}")
        if rot % 16 or not 16 <= rot <= 256:
            raise ValueError("rot must be a multiple of 16 in 16 .. 256")
        self.rot, self.layout = int(rot), layout
        n = self.rot // 2
        freqs, mag = (ctypes.c_double * n)(), ctypes.c_double(1.0)
        lib = _lib.load()
        if inv_freq is None:
            if magnitude is not None:
                raise ValueError("magnitude goes with inv_freq")
            _lib.check("gqa_attn_rope_freqs",
                       lib.gqa_attn_rope_freqs(self.rot, float(base), SCALINGS[scaling], float(factor),
                                               int(original_length or 0), float(beta_fast), float(beta_slow), freqs,
                                               ctypes.byref(mag)))
        else:
            values = [float(f) for f in inv_freq]
            if len(values) != n:
                raise ValueError(f"inv_freq must hold rot / 2 = {n} numbers")
            freqs[:] = values
            mag.value = 1.0 if magnitude is None else float(magnitude)
        words = (ctypes.c_uint64 * n)()
        _lib.check("gqa_attn_rope_turns", lib.gqa_attn_rope_turns(freqs, n, words))
        self.inv_freq, self.magnitude = list(freqs), mag.value
        self._words = torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64)
        self._on = {}
        if device is not None:
            self.on(device)

    def on(self, device) -> torch.Tensor:
        """The words on ``device`` (copied once)."""
        dev = _device(device)
        if dev not in self._on:
            self._on[dev] = self._words.to(dev)
        return self._on[dev]

    def struct(self, device, positions, pos_offset) -> _lib.Rope:
        words = self._on.get(device)
        if words is None:
            words = self.on(device)
        return _lib.Rope(words.data_ptr(), None if positions is None else positions.data_ptr(),
                         0 if positions is None or positions.dim() == 1 else positions.stride(0), pos_offset,
                         self.magnitude, self.rot, LAYOUTS[self.layout])


def rotate(q, k, table, *, positions=None, pos_offset=0, inverse=False, out=None, out_k=None, stream=None):
    """Rotated ``(q, k)`` in one launch; ``k`` may be ``None``.  Positions are
    ``pos_offset + l``, or ``positions`` (int32, [L] or [B, L]).  ``inverse`` turns back by
    the same angles (with the same magnitude: the gradient of the rotation).  ``out`` /
    ``out_k`` may be given and may be ``q`` / ``k`` themselves.  Asynchronous on ``stream``."""
    if not (isinstance(q, torch.Tensor) and q.is_cuda and q.dim() == 4):
        raise ValueError("rotate takes 4-d CUDA tensors")
    dev, dtype = q.device, q.dtype
    code = float_code(dtype)
    B, _, L, d = q.shape
    rq = rows(q, "q", dev, dtype)
    positions = check_positions(positions, B, L, dev)
    if positions is not None and pos_offset:
        raise ValueError("pos_offset goes with positions counted from it, not with positions given")
    if k is not None and (k.dim() != 4 or k.shape[0] != B or k.shape[2] != L or k.shape[3] != d):
        raise ValueError("k must be [B, Hkv, L, 256] with q's B and L")
    if k is None and out_k is not None:
        raise ValueError("out_k needs k")
    with on_stream(stream):
        out = new_like(q) if out is None else out
        if k is not None and out_k is None:
            out_k = new_like(k)
    if out.shape != q.shape or (k is not None and out_k.shape != k.shape):
        raise ValueError("out must have the shape of its input")
    ro = rows(out, "out", dev, dtype, written=True)
    rk = ok = None
    if k is not None:
        rk, ok = ctypes.byref(rows(k, "k", dev, dtype)), ctypes.byref(rows(out_k, "out_k", dev, dtype, written=True))
    launch("gqa_attn_rope", dev, stream, ctypes.byref(rq), ctypes.byref(ro), rk, ok, B, L, d, code,
           ctypes.byref(table.struct(dev, positions, int(pos_offset))), int(bool(inverse)))
    return out, out_k


class _Rotate(torch.autograd.Function):
    """rotate as the forward, the inverse rotation of the gradients as the backward, itself
    differentiable: the rotation is linear, so that is right to any order."""

    @staticmethod
    def forward(ctx, q, k, table, positions, pos_offset, inverse):
        ctx.table, ctx.pos_offset, ctx.inverse = table, pos_offset, inverse
        ctx.save_for_backward(positions)
        ctx.set_materialize_grads(False)  # an output that the loss does not use has no gradient, not one of zeros
        out, out_k = rotate(q, k, table, positions=positions, pos_offset=pos_offset, inverse=inverse)
        return out if k is None else (out, out_k)

    @staticmethod
    def backward(ctx, dq, dk=None):
        (positions,) = ctx.saved_tensors
        dq = _dense_rows(dq) if ctx.needs_input_grad[0] else None
        dk = _dense_rows(dk) if ctx.needs_input_grad[1] else None

        def back(a, b):
            if torch.is_grad_enabled():  # create_graph
                got = _Rotate.apply(a, b, ctx.table, positions, ctx.pos_offset, not ctx.inverse)
                return (got, None) if b is None else got
            return rotate(a, b, ctx.table, positions=positions, pos_offset=ctx.pos_offset, inverse=not ctx.inverse)

        if dq is not None:
            dq, dk = back(dq, dk)
        elif dk is not None:
            dk, _ = back(dk, None)
        return dq, dk, None, None, None, None


def _dense_rows(g):
    """A gradient as ``rotate`` takes it: autograd may hand in expanded or sliced ones, and dense
    ones that start anywhere (a part of a concatenated tensor's), which are contiguous as they are."""
    if g is None:
        return None
    unit = 16 // g.element_size()
    whole = g.stride(3) == 1 and all(s % unit == 0 for s in g.stride()[:3]) and g.data_ptr() % 16 == 0
    return g if whole else g.clone(memory_format=torch.contiguous_format)


def rotate_autograd(q, k, table, *, positions=None, pos_offset=0):
    """Differentiable ``rotate`` (new tensors), to any order; ``k`` may be ``None``.  The
    positions carry no gradient."""
    if k is None:
        return _Rotate.apply(q, None, table, positions, int(pos_offset), False), None
    return _Rotate.apply(q, k, table, positions, int(pos_offset), False)
