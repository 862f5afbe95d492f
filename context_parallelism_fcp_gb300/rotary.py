"""Rotary positions of include/fcp.h: of q and k for the attention over a work list, and of a batch's new
tokens on their way to a paged cache. As in the rest of the package the arguments are checked and
marshalled here and all the work is done by the library's kernels."""
from __future__ import annotations

import ctypes
import math
from fractions import Fraction
from typing import Optional, Sequence, Tuple

import numpy as np
import torch

from . import _check, _RotaryStruct, _stream, lib
from .paged import CacheBatch, PagedCache, _here, _Owner, _want

__all__ = ["Rotary", "rotary_apply", "rotary_backward", "rotary_write"]


def frequencies(rotary_dim: int, base: float = 10000.0, scaling: Optional[dict] = None) -> Tuple[np.ndarray, float]:
    """(radians a position of each pair in float64, factor of the turned pairs). f_i = base^(-2 i / rotary_dim);
    ``scaling`` stretches it for contexts ``factor`` times as long as the ``original`` one of training:

    * kind "linear": f / factor;
    * "ntk": base * factor^(rotary_dim / (rotary_dim - 2)), so that the slowest pair is stretched by factor
      and the fastest stays;
    * "yarn": pairs that turn more than ``fast`` (32) times over the original context stay, those that
      turn less than ``slow`` (once) are divided by factor, in between by a ramp over the pairs; the factor of
      the turned pairs is ``magnitude``, 0.1 ln(factor) + 1 unless given;
    * "bands": the same with wavelengths, f / factor below ``slow`` (1) turns over the original context, f above
      ``fast`` (4) turns, and a ramp over the number of turns in between.
    """
    half = rotary_dim // 2
    i = np.arange(half, dtype=np.float64)
    scaling = dict(scaling or {"kind": None})
    kind, magnitude = scaling.pop("kind", None), 1.0

    def need(*names, **defaults):
        values = [scaling.pop(n, None) for n in names] + [scaling.pop(n, d) for n, d in defaults.items()]
        if scaling or any(v is None for v in values[:len(names)]):
            raise ValueError(f"scaling {kind!r} takes {', '.join([*names, *defaults])}")
        for n, v in zip([*names, *defaults], values):
            if v is not None and not (float(v) > 0 and math.isfinite(float(v))):
                raise ValueError(f"scaling {kind!r}: {n} must be positive, got {v}")
        return [None if v is None else float(v) for v in values]

    if kind == "ntk":
        (factor,) = need("factor")
        if rotary_dim <= 2:
            raise ValueError("scaling 'ntk' needs more than one pair")
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = base ** (-2.0 * i / rotary_dim)
    if kind == "linear":
        (factor,) = need("factor")
        f = f / factor
    elif kind == "yarn":
        factor, original, fast, slow, magnitude = need("factor", "original", fast=32.0, slow=1.0, magnitude=None)
        low, high = (rotary_dim * math.log(original / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (fast, slow))
        # the upper end may lie past the last pair, which then keeps a part of its frequency
        low, high = max(math.floor(low), 0), min(math.ceil(high), rotary_dim - 1)
        ramp = np.clip((i - low) / max(high - low, 0.001), 0.0, 1.0)
        f = f * (1 - ramp) + f / factor * ramp
        if magnitude is None:
            magnitude = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    elif kind == "bands":
        factor, original, slow, fast = need("factor", "original", slow=1.0, fast=4.0)
        if fast <= slow:
            raise ValueError("scaling 'bands': fast must be larger than slow")
        keep = np.clip((original * f / (2 * math.pi) - slow) / (fast - slow), 0.0, 1.0)
        f = f * keep + f / factor * (1 - keep)
    elif kind not in (None, "ntk"):
        raise ValueError(f"scaling's kind must be linear, ntk, yarn or bands, got {kind!r}")
    elif kind is None and scaling:
        raise ValueError("scaling needs a kind")
    return f, magnitude


def turns(radians: Sequence[float]) -> np.ndarray:
    """Radians a position as turns a position in units of 2^-64 (uint64): the nearest integer, whole turns
    left out."""
    # pi to 36 digits, twice what float64 holds: the quotient is right to the unit
    pi = Fraction(3141592653589793238462643383279502884, 10 ** 36)
    return np.array([round(Fraction(float(x)) / (2 * pi) * 2 ** 64) % 2 ** 64 for x in radians], dtype=np.uint64)


class Rotary(_Owner):
    """The frequencies of rotary positions on the device (fcp_rotary): the first ``rotary_dim`` channels of
    a head are turned, in pairs rotary_dim / 2 apart, or neighbours (``interleaved``). ``base`` and ``scaling``
    as in ``frequencies``; or ``radians``, one value a pair, and ``magnitude``, given outright."""

    def __init__(self, rotary_dim: int, base: float = 10000.0, interleaved: bool = False, scaling: Optional[dict] = None,
                 radians: Optional[Sequence[float]] = None, magnitude: Optional[float] = None, device="cuda"):
        rotary_dim = int(rotary_dim)
        if rotary_dim <= 0 or rotary_dim > 128 or rotary_dim % 16:
            raise ValueError(f"rotary_dim must be a multiple of 16 up to 128, got {rotary_dim}")
        if not (base > 1 and math.isfinite(base)):
            raise ValueError(f"base must be larger than 1, got {base}")
        if radians is None:
            radians, size = frequencies(rotary_dim, float(base), scaling)
        elif scaling is not None:
            raise ValueError("radians are given: no scaling")
        else:
            radians, size = np.asarray(radians, dtype=np.float64), 1.0
        if radians.shape != (rotary_dim // 2,) or not np.isfinite(radians).all():
            raise ValueError(f"radians must be {rotary_dim // 2} finite numbers")
        self.magnitude = float(size if magnitude is None else magnitude)
        if not (self.magnitude > 0 and self.magnitude < 3e38):
            raise ValueError(f"magnitude must be positive, got {magnitude}")
        self.rotary_dim, self.interleaved, self.radians = rotary_dim, bool(interleaved), radians
        self.turns = torch.from_numpy(turns(radians).view(np.int64)).to(device)
        if self.turns.device.type != "cuda":
            raise ValueError("the frequencies must be on a CUDA device")
        self._own([self.turns], self.turns.get_device())
        self._struct = _RotaryStruct(self.turns.data_ptr(), self.magnitude, rotary_dim, int(self.interleaved))
        self._ref = ctypes.byref(self._struct)


def _outlike(x, stream):
    """A tensor like x, as memory of the stream that the call runs on."""
    if stream is not None and not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_stream(stream), device=x.device)
    with torch.cuda.stream(stream):
        return torch.empty_like(x)


def _apply(rotary: Rotary, q, k, positions, q_out, k_out, stream, backward: int):
    index = rotary._index
    raw = _here(index, stream, "frequencies")
    one = k if q is None else q
    if not isinstance(one, torch.Tensor) or one.dim() != 3 or (k is not None and (not isinstance(k, torch.Tensor) or k.dim() != 3)):
        raise ValueError("q and k must be tensors [heads, T, D], one of them at least")
    _, T, D = one.shape
    _want(positions, torch.int32, (T,), index, "positions", "frequencies")
    hq = hkv = 0
    if q is not None:
        hq, shape = q.shape[0], q.shape
        _want(q, torch.bfloat16, shape, index, "q", "frequencies")
        if q_out is None:
            q_out = _outlike(q, stream)
        else:
            _want(q_out, torch.bfloat16, shape, index, "q_out", "frequencies")
    elif q_out is not None:
        raise ValueError("q_out without q")
    if k is not None:
        hkv, shape = k.shape[0], (k.shape[0], T, D)
        _want(k, torch.bfloat16, shape, index, "k", "frequencies")
        if k_out is None:
            k_out = _outlike(k, stream)
        else:
            _want(k_out, torch.bfloat16, shape, index, "k_out", "frequencies")
    elif k_out is not None:
        raise ValueError("k_out without k")
    if raw not in rotary._streams:
        rotary._note(raw, stream)
    status = lib().fcp_rotary_apply(rotary._ref, positions.data_ptr(), T, q.data_ptr() if hq else None,
                                    q_out.data_ptr() if hq else None, hq, k.data_ptr() if hkv else None,
                                    k_out.data_ptr() if hkv else None, hkv, D, backward, raw)
    if status:
        _check(status, "fcp_rotary_apply")
    return q_out, k_out


def rotary_apply(rotary: Rotary, q, k, positions, q_out=None, k_out=None, stream=None):
    """(q, k) turned by their rows' positions (fcp_rotary_apply): q [Hq, T, D] and k [Hkv, T, D] in bf16,
    either of them None, positions int32 [T]. q_out and k_out may be q and k; they are allocated unless
    given (as memory of the stream that the call runs on)."""
    return _apply(rotary, q, k, positions, q_out, k_out, stream, 0)


def rotary_backward(rotary: Rotary, dq, dk, positions, dq_out=None, dk_out=None, stream=None):
    """The gradients of rotary_apply's q and k from those of what it returned."""
    return _apply(rotary, dq, dk, positions, dq_out, dk_out, stream, 1)


def rotary_write(cache: PagedCache, batch: CacheBatch, rotary: Rotary, q, k, v, q_out=None, stream=None):
    """The new tokens' q and k turned by their positions in their sequences, and the turned k and v written
    to the cache (fcp_rotary_write). q [Hq, total_new, D] may be None. Returns the turned q: q_out, which may
    be q, and is allocated unless given (rows of no sequence are undefined then, and otherwise left as they
    were)."""
    index = cache._index
    if batch._index != index or rotary._index != index:
        raise ValueError("the batch, the frequencies and the cache must be on one device")
    shape = (cache.hkv, batch.total_new, cache.head_dim)
    _want(k, torch.bfloat16, shape, index, "k")
    _want(v, torch.bfloat16, shape, index, "v")
    raw = _here(index, stream)
    hq = 0
    if q is not None:
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("q must be a tensor [Hq, total_new, D]")
        hq = q.shape[0]
        _want(q, torch.bfloat16, (hq, *shape[1:]), index, "q")
        if q_out is None:
            q_out = _outlike(q, stream)
        else:
            _want(q_out, torch.bfloat16, (hq, *shape[1:]), index, "q_out")
    elif q_out is not None:
        raise ValueError("q_out without q")
    if raw not in cache._streams:
        cache._note(raw, stream)
    if raw not in rotary._streams:
        rotary._note(raw, stream)
    if batch._pool is not None and raw not in batch._pool._streams:
        batch._pool._note(raw, stream)
    status = lib().fcp_rotary_write(cache._ref, batch._ref, rotary._ref, q.data_ptr() if hq else None,
                                    q_out.data_ptr() if hq else None, hq, k.data_ptr(), v.data_ptr(), raw)
    if status:
        _check(status, "fcp_rotary_write")
    return q_out
