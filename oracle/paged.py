"""The paged cache and its attention in float64 numpy, from their definitions: one sequence and
one head at a time, no pages beyond looking a row up, nothing shared with the library."""
from __future__ import annotations

import math
from typing import List, Tuple

import numpy as np


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 e4m3 codes (sign, 4 exponent bits with bias 7, 3 mantissa bits;
    0x7f and 0xff are NaN)."""
    out = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.nan if c & 0x7F == 0x7F else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        out[c] = -x if c & 0x80 else x
    return out


_FINITE = np.sort(e4m3_values()[:0x7F])  # codes 0 .. 0x7e in increasing order, code = index


def quantise_row(x: np.ndarray) -> Tuple[np.ndarray, int]:
    """(codes, scale byte) of one row: k the smallest integer >= -126 with max|x| <= 448 * 2^k, the
    codes those nearest to x / 2^k, ties to the even code, of those whose value bf16 holds (256 * 2^120
    is 2^128: the only one it does not)."""
    if not np.isfinite(x).all():
        return np.zeros(x.shape, np.uint8), 255
    top = float(np.abs(x).max())
    k = 0
    if top > 0:
        k = -126
        while top > 448.0 * 2.0 ** k:
            k += 1
    y = np.minimum(np.abs(x) / 2.0 ** k, 240.0 if k == 120 else 448.0)
    hi = np.clip(np.searchsorted(_FINITE, y), 0, 0x7E)
    lo = np.maximum(hi - 1, 0)
    d_hi, d_lo = _FINITE[hi] - y, y - _FINITE[lo]
    code = np.where((d_lo < d_hi) | ((d_lo == d_hi) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    return code | (np.signbit(x).astype(np.uint8) << 7), k + 127


def row_value(codes: np.ndarray, byte: int) -> np.ndarray:
    return e4m3_values()[codes] * (math.nan if byte == 255 else 2.0 ** (byte - 127))


def places(new: List[int], lens: List[int], table: np.ndarray, page: int):
    """(packed row, sequence, position, page, row of the page) of every new token whose position is
    not negative."""
    row = 0
    for i, (n, length) in enumerate(zip(new, lens)):
        for j in range(n):
            pos = length - n + j
            if pos >= 0:
                yield row + j, i, pos, int(table[i, pos // page]), pos % page
        row += n


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, n: int, causal: bool):
    """One sequence and query head: q [n, D] against its rows k, v [len, D]. Returns o, lse and, for
    error bounds, sum_j w_j |v_j|, sqrt(sum_j w_j^2 v_j^2) and max_j sum_c |q_c k_jc| / sqrt(D)."""
    d, length = q.shape[1], k.shape[0]
    o, lse = np.zeros((n, d)), np.full(n, -np.inf)
    spread, rms, size = np.zeros((n, d)), np.zeros((n, d)), np.zeros(n)
    for j in range(n):
        seen = length - n + j + 1 if causal else length
        if seen <= 0:
            continue
        s = k[:seen] @ q[j] / math.sqrt(d)
        top = s.max()
        w = np.exp(s - top)
        total = w.sum()
        w /= total
        o[j], lse[j] = w @ v[:seen], top + math.log(total)
        spread[j], rms[j] = w @ np.abs(v[:seen]), np.sqrt((w * w) @ (v[:seen] ** 2))
        size[j] = (np.abs(k[:seen]) @ np.abs(q[j])).max() / math.sqrt(d)
    return o, lse, spread, rms, size
