"""The ramp of yarn's scaling against its definition, worked out pair by pair, with no GPU: also over contexts so long
that the slowest pair of channels turns more than once, where the ramp ends past the last pair."""
import math

import numpy as np
import pytest

CASES = [(64, 10000.0, 4096, 16.0), (128, 500000.0, 8192, 8.0), (128, 10000.0, 32768, 4.0),   # the last pair is behind the ramp
         (128, 10000.0, 65536, 4.0), (128, 10000.0, 131072, 4.0), (16, 10000.0, 32768, 16.0),  # or inside it
         (32, 10000.0, 100000, 2.0), (96, 500.0, 4096, 32.0),
         (64, 10000.0, 1 << 22, 8.0), (128, 10000.0, 1 << 40, 8.0)]                             # or before it


def factors(dim, base, original, fast, slow):
    """How much of each pair's frequency is kept as it is, 1 to 0. Pair x turns original / (2 pi) * base^(-2 x / dim)
    times over the original context; the ramp begins at the last whole x where that is `fast` at least, and ends
    at the first where it is `slow` at most."""
    turns = lambda x: original / (2 * math.pi) * base ** (-2.0 * x / dim)  # noqa: E731
    begin = max((x for x in range(4 * dim) if turns(x) >= fast), default=0)
    end = min(x for x in range(4 * dim) if turns(x) <= slow)
    return [min(max((end - x) / (end - begin), 0.0), 1.0) for x in range(dim // 2)], turns


@pytest.mark.parametrize("dim,base,original,factor", CASES, ids=str)
def test_the_ramp_is_the_definitions(fcp, dim, base, original, factor):
    from context_parallelism_fcp_gb300 import rotary

    plain = rotary.frequencies(dim, base)[0]
    got = rotary.frequencies(dim, base, dict(kind="yarn", factor=factor, original=original))[0]
    keep, turns = factors(dim, base, original, 32.0, 1.0)
    want = plain * (np.array(keep) + (1 - np.array(keep)) / factor)
    assert np.allclose(got, want, rtol=1e-12, atol=0)
    for x in range(dim // 2):  # what the function says of itself
        if turns(x) > 32:
            assert got[x] == plain[x]
        if turns(x) > 1:
            assert got[x] > plain[x] / factor * (1 + 1e-9), x
        elif x >= min(y for y in range(4 * dim) if turns(y) <= 1):
            assert math.isclose(got[x], plain[x] / factor, rel_tol=1e-14)


@pytest.mark.parametrize("fast,slow", [(8.0, 0.5), (64.0, 2.0), (4.0, 3.9)])
def test_other_ends(fcp, fast, slow):
    from context_parallelism_fcp_gb300 import rotary

    dim, base, original, factor = 128, 10000.0, 200000, 16.0
    plain = rotary.frequencies(dim, base)[0]
    got = rotary.frequencies(dim, base, dict(kind="yarn", factor=factor, original=original, fast=fast, slow=slow))[0]
    keep = np.array(factors(dim, base, original, fast, slow)[0])
    assert np.allclose(got, plain * (keep + (1 - keep) / factor), rtol=1e-12, atol=0)
