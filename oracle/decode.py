"""Decoding from a cache in float64: rotary positions, quantised rows, drafted tokens.

Test infrastructure (see the package docstring): never imported by the product.

* ``rotate``: pair (x1, x2) at position p turns by a = p f_i,
  y1 = m (x1 cos a - x2 sin a), y2 = m (x2 cos a + x1 sin a).  The angle's fraction of a
  turn is taken in exact integer arithmetic (positions are whole numbers and f_i is a
  binary fraction), so far positions lose nothing.
* ``quantise``: the least power of two s with amax / s <= 448 over the finite values of
  a row, and the nearest numbers of three mantissa bits (ties to even, least exponent
  -6, largest 448) to x / s.
* ``tree_attention``: attention of drafted tokens behind a context (system1-omni issue
  #27, item 3: a state computed once, then what follows it), one sequence at a time, only
  over the keys that a row sees.
"""

from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

from .exact import _as_f64

# pi to 50 digits, as a ratio of whole numbers (the fraction of a turn needs p f / (2 pi)).
_PI = Fraction(314159265358979323846264338327950288419716939937511, 10 ** 50)


def angle(position: int, frequency: float) -> float:
    """position * frequency reduced to one turn around zero, in float64."""
    turns = Fraction(frequency) * int(position) / (2 * _PI)
    turns -= math.floor(turns)
    if turns > Fraction(1, 2):
        turns -= 1
    return float(turns * 2 * _PI)


def rotate(x, positions, inv_freq, magnitude=1.0, layout="half", sign=1.0):
    """x [B, H, L, d], positions [B, L] (whole numbers) -> rotated float64 array."""
    x = _as_f64(x)
    R = 2 * len(inv_freq)
    a = np.array([[[angle(p, f) for f in inv_freq] for p in row] for row in np.asarray(positions)])
    c, s = magnitude * np.cos(a)[:, None], sign * magnitude * np.sin(a)[:, None]
    y = x.copy()
    lo, hi = (slice(0, R // 2), slice(R // 2, R)) if layout == "half" else (slice(0, R, 2), slice(1, R, 2))
    y[..., lo] = x[..., lo] * c - x[..., hi] * s
    y[..., hi] = x[..., hi] * c + x[..., lo] * s
    return y


def quantise(x):
    """(codes' values, scale) of rows [..., d]: values are on the e4m3 grid, x ~ value * scale."""
    x = _as_f64(x)
    finite = np.where(np.isfinite(x), np.abs(x), 0.0)
    amax = finite.max(-1)
    scale = np.ones_like(amax)
    for i in np.ndindex(amax.shape):
        if amax[i] > 0:
            m, e = math.frexp(amax[i] / 448.0)
            scale[i] = 2.0 ** min(120, max(-120, e - 1 if m == 0.5 else e))
    y = x / scale[..., None]
    with np.errstate(invalid="ignore"):
        _, e = np.frexp(np.where(np.isfinite(y), y, 1.0))
        step = 2.0 ** (np.maximum(e - 1, -6) - 3.0)
        y = np.clip(np.rint(y / step) * step, -448.0, 448.0)
    return y, scale


def tree_attention(q, k, v, context, drafted, mask=None):
    """One sequence: q [Hq, T, d], k / v [Hkv, >= context + drafted, d]; ``mask`` [T, T] of
    truth values or None (a chain).  Returns (out, lse, spread) with spread the
    probability-weighted sum of |v|, the size that errors of probabilities act on."""
    q, k, v = _as_f64(q), _as_f64(k), _as_f64(v)
    Hq, T, d = q.shape
    G = Hq // k.shape[0]
    size = np.abs(v)
    out, spread, lse = np.zeros((Hq, T, d)), np.zeros((Hq, T, d)), np.full((Hq, T), -np.inf)
    for t in range(min(T, drafted)):
        seen = [context + u for u in range(drafted) if (u <= t if mask is None else mask[t][u])]
        if context + len(seen) == 0:
            continue
        for g in range(k.shape[0]):
            h = slice(g * G, (g + 1) * G)
            # the context's rows are used in place, the drafted ones that the row sees are picked out
            s = np.concatenate([q[h, t] @ k[g, :context].T, q[h, t] @ k[g, seen].T], axis=1) / math.sqrt(d)
            top = s.max(1, keepdims=True)
            p = np.exp(s - top)
            total = p.sum(1, keepdims=True)
            p /= total
            out[h, t] = p[:, :context] @ v[g, :context] + p[:, context:] @ v[g, seen]
            spread[h, t] = p[:, :context] @ size[g, :context] + p[:, context:] @ size[g, seen]
            lse[h, t] = (top + np.log(total))[:, 0]
    return out, lse, spread
