"""Rotary positions with no GPU: frequencies, their integers, refusals, and the oracle's gradient."""
import ctypes
import math

import numpy as np
import pytest

from oracle import rotary as R

INVALID, UNSUPPORTED = 1, 3
P = 1 << 12  # an aligned address that is never looked at


@pytest.fixture(scope="module")
def rot(fcp):
    from context_parallelism_fcp_gb300 import rotary

    return rotary


def test_frequencies(rot):
    f, m = rot.frequencies(8, 16.0)
    assert m == 1.0 and np.allclose(f, [1, 0.5, 0.25, 0.125], rtol=1e-15)
    assert np.allclose(rot.frequencies(8, 16.0, dict(kind="linear", factor=4))[0], f / 4, rtol=1e-15)
    ntk, m = rot.frequencies(8, 16.0, dict(kind="ntk", factor=4))
    assert m == 1.0 and ntk[0] == 1.0 and math.isclose(ntk[3], f[3] / 4, rel_tol=1e-14)
    yarn, m = rot.frequencies(64, 10000.0, dict(kind="yarn", factor=16, original=4096))
    plain = rot.frequencies(64)[0]
    assert math.isclose(m, 0.1 * math.log(16) + 1) and np.allclose(yarn[:10], plain[:10], rtol=1e-15)
    assert np.allclose(yarn[-8:], plain[-8:] / 16, rtol=1e-14) and (np.diff(yarn) < 0).all()
    assert rot.frequencies(64, 10000.0, dict(kind="yarn", factor=16, original=4096, magnitude=1.5))[1] == 1.5
    bands, m = rot.frequencies(64, 500000.0, dict(kind="bands", factor=8, original=8192))
    plain = rot.frequencies(64, 500000.0)[0]
    turns = 8192 * plain / (2 * math.pi)
    assert m == 1.0 and np.allclose(bands[turns >= 4], plain[turns >= 4]) and np.allclose(bands[turns <= 1], plain[turns <= 1] / 8)
    between = (turns > 1) & (turns < 4)
    assert between.any() and ((bands < plain) & (bands > plain / 8))[between].all()


@pytest.mark.parametrize("scaling", [dict(kind="other"), dict(kind="linear"), dict(kind="linear", factor=-1),
                                     dict(kind="yarn", factor=2), dict(kind="linear", factor=2, original=3), dict(factor=2),
                                     dict(kind="bands", factor=2, original=8, fast=1, slow=1),
                                     dict(kind="ntk", factor=float("nan"))], ids=str)
def test_scalings_that_are_refused(rot, scaling):
    with pytest.raises(ValueError):
        rot.frequencies(64, 10000.0, scaling)


def test_turns(rot):
    assert rot.turns([0.0, 2 * math.pi * 0.0]).tolist() == [0, 0]
    t = rot.turns([1.0, math.pi, -1.0, 1e-12])
    assert t[0] == round(2 ** 64 / (2 * math.pi), -4) or abs(int(t[0]) - 2 ** 64 / (2 * math.pi)) < 2 ** 12
    assert abs(int(t[1]) - 2 ** 63) < 2 ** 11 and (int(t[0]) + int(t[2])) % 2 ** 64 == 0
    assert int(t[3]) == round(1e-12 / (2 * math.pi) * 2 ** 64)


def test_the_oracles_gradient_against_differences():
    rng = np.random.default_rng(0)
    for interleaved in (False, True):
        x, g = rng.normal(size=(2, 2, 5, 64))
        pos, f = np.array([0, 1, 7, -3, 100000]), 10.0 ** -rng.random(16)
        grad = R.turn(g, pos, f, 1.3, interleaved, backward=True)[0]
        loss = lambda y: (R.turn(y, pos, f, 1.3, interleaved)[0] * g).sum()  # noqa: E731
        for at in [(0, 0, 0), (1, 2, 16), (0, 4, 31), (1, 3, 5), (0, 4, 50)]:
            y = x.copy()
            y[at] += 0.5
            up = loss(y)
            y[at] -= 1.0
            assert abs(up - loss(y) - grad[at]) < 1e-9


def _struct(**change):
    from context_parallelism_fcp_gb300 import _RotaryStruct

    return _RotaryStruct(**{**dict(turns=P, magnitude=1.0, rotary_dim=64, interleaved=0), **change})


@pytest.mark.parametrize("change,status", [(dict(turns=None), INVALID), (dict(turns=P + 4), INVALID), (dict(magnitude=0.0), INVALID),
                                           (dict(magnitude=float("inf")), INVALID), (dict(magnitude=float("nan")), INVALID),
                                           (dict(rotary_dim=0), INVALID), (dict(rotary_dim=80), INVALID),
                                           (dict(rotary_dim=24), UNSUPPORTED)], ids=str)
def test_both_calls_refuse(fcp, change, status):
    from context_parallelism_fcp_gb300 import _CacheBatchStruct, _CacheStruct

    L = fcp.lib()
    r = ctypes.byref(_struct(**change))
    c = _CacheStruct(k_pages=P, v_pages=P, status=P, n_pages=4, hkv=2, page_size=16, head_dim=64)
    b = _CacheBatchStruct(cu_new=P, lens=P, block_table=P, n_seqs=2, max_pages=3, total_new=5, max_new=4)
    assert L.fcp_rotary_apply(r, P, 5, P, P, 4, P, P, 2, 64, 0, None) == status
    assert L.fcp_rotary_write(ctypes.byref(c), ctypes.byref(b), r, P, P, 4, P, P, None) == status


def test_buffers_and_sizes(fcp):
    from context_parallelism_fcp_gb300 import _CacheBatchStruct, _CacheStruct

    L = fcp.lib()
    good = [ctypes.byref(_struct()), P, 5, P, P, 4, P, P, 2, 64, 0, None]
    for at, value, status in ((0, None, INVALID), (1, None, INVALID), (1, P + 2, INVALID), (2, -1, INVALID), (3, None, INVALID),
                              (3, P + 8, INVALID), (4, None, INVALID), (5, -1, INVALID), (6, None, INVALID), (7, P + 4, INVALID),
                              (8, -1, INVALID), (9, 96, UNSUPPORTED), (2, (1 << 30) + 1, UNSUPPORTED), (5, 65536, UNSUPPORTED)):
        args = list(good)
        args[at] = value
        assert L.fcp_rotary_apply(*args) == status, (at, value)
    nothing = list(good)
    nothing[1:9] = [None, 0, None, None, 4, None, None, 2]
    assert L.fcp_rotary_apply(*nothing) == 0
    nothing[1:9] = [None, 5, None, None, 0, None, None, 0]
    assert L.fcp_rotary_apply(*nothing) == 0
    c = _CacheStruct(k_pages=P, v_pages=P, status=P, n_pages=4, hkv=2, page_size=16, head_dim=64)
    b = _CacheBatchStruct(cu_new=P, lens=P, block_table=P, n_seqs=2, max_pages=3, total_new=5, max_new=4)
    good = [ctypes.byref(c), ctypes.byref(b), ctypes.byref(_struct()), P, P, 4, P, P, None]
    for at, value in ((0, None), (1, None), (2, None), (3, None), (4, P + 8), (5, -1), (6, None), (7, P + 2)):
        args = list(good)
        args[at] = value
        assert L.fcp_rotary_write(*args) == INVALID, (at, value)
    b0 = _CacheBatchStruct(n_seqs=0, max_pages=0, total_new=0, max_new=0)
    assert L.fcp_rotary_write(ctypes.byref(c), ctypes.byref(b0), ctypes.byref(_struct()), None, None, 4, None, None, None) == 0


@pytest.mark.parametrize("how", [dict(rotary_dim=24), dict(rotary_dim=0), dict(rotary_dim=144), dict(rotary_dim=64, base=1.0),
                                 dict(rotary_dim=64, radians=[1.0] * 31), dict(rotary_dim=16, radians=[1.0] * 7 + [math.inf]),
                                 dict(rotary_dim=16, radians=[1.0] * 8, scaling=dict(kind="linear", factor=2)),
                                 dict(rotary_dim=64, magnitude=0.0), dict(rotary_dim=64)], ids=str)
def test_the_binding_refuses(fcp, how):
    with pytest.raises(ValueError):
        fcp.Rotary(**how, device="cpu")  # the last one for its device
    assert {"Rotary", "rotary_apply", "rotary_backward", "rotary_write"} <= set(fcp.__all__)
