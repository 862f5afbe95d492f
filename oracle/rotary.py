"""Rotary positions in float64 numpy, from their definition: nothing shared with the library."""
from __future__ import annotations

import numpy as np


def pairs(part: int, interleaved: bool):
    """(a, b) channels of every pair."""
    i = np.arange(part // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + part // 2)


def turn(x: np.ndarray, positions: np.ndarray, radians: np.ndarray, magnitude: float, interleaved: bool,
         backward: bool = False):
    """x [..., T, D] with the first 2 len(radians) channels turned, and for error bounds m (|a| + |b|) of each
    channel's pair (0 for the others). Angles in long double, reduced there."""
    angle = np.fmod(positions.astype(np.longdouble)[:, None] * radians.astype(np.longdouble), 8 * np.arctan(np.longdouble(1)))
    c, s = (magnitude * f(angle).astype(np.float64) for f in (np.cos, np.sin))
    if backward:
        s = -s
    a, b = pairs(2 * len(radians), interleaved)
    y, size = x.astype(np.float64).copy(), np.zeros(x.shape)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    size[..., a] = size[..., b] = magnitude * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y, size
