"""Rows of a 4-bit cache in float64 numpy, from their definition: e2m1 codes, an e4m3 scale for every
16 channels and a power-of-two unit; nothing shared with the library."""
from __future__ import annotations

import math
from typing import Tuple

import numpy as np

from .paged import e4m3_values

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
_SCALES = e4m3_values()[:0x7F]  # codes 0 .. 0x7e in increasing order


def _nearest(y: np.ndarray, values: np.ndarray) -> np.ndarray:
    """Indices of the nearest of increasing `values`, the even index at ties."""
    hi = np.clip(np.searchsorted(values, y), 0, len(values) - 1)
    lo = np.maximum(hi - 1, 0)
    d_hi, d_lo = values[hi] - y, y - values[lo]
    return np.where((d_lo < d_hi) | ((d_lo == d_hi) & (lo % 2 == 0)), lo, hi)


def quantise(x: np.ndarray, unit: float) -> Tuple[np.ndarray, np.ndarray]:
    """Rows [..., D] as (codes [..., D] from 0 to 15, scale bytes [..., D / 16])."""
    y = x.reshape(*x.shape[:-1], -1, 16) / unit
    ok = np.isfinite(y).all(-1)
    y = np.where(ok[..., None], y, 0.0)
    byte = np.maximum(_nearest(np.minimum(np.abs(y).max(-1) / 6, 448.0), _SCALES), 1)
    code = _nearest(np.minimum(np.abs(y) / _SCALES[byte][..., None], 6.0), E2M1)
    code = np.where(np.signbit(y), code + 8, code)
    return code.reshape(x.shape), np.where(ok, byte, 0x7F)


def value(codes: np.ndarray, bytes_: np.ndarray, unit: float) -> np.ndarray:
    """What codes [..., D] with their scale bytes [..., D / 16] stand for."""
    x = np.where(codes >= 8, -1.0, 1.0) * E2M1[codes % 8]
    scale = np.where(bytes_ == 0x7F, math.nan, np.append(_SCALES, math.nan)[bytes_ & 0x7F]) * unit
    return x * np.repeat(scale, 16, -1)


def unpack(packed: np.ndarray) -> np.ndarray:
    """Codes [..., D] of bytes [..., D / 2], the even channel in the low half."""
    return np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], -1)
