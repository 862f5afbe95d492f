"""How exact the attention over a 4-bit cache is said to be, held to that: P rounded to f16.

A weight is rounded by at most 2^-11 of itself, or by 2^-32 of the row's largest: weights are held relative to the running
maximum so that the largest is 2^7 at least, and f16 numbers below 2^-14 are multiples of 2^-24, off by half of that. The
sum of the weights is float32 and not rounded. Scores are float32 sums of D exact products, off by D 2^-24 of the sum of
their magnitudes, which is how much their weight is off, of itself; the sum of the weights once more. The products
with V are added 16 keys at a time, some 250 times for 4000 keys, each sum off by 2^-23 of what is there: 2^-15; exp2, the
running sum and the joins are below that together. So an element of o is off by at most

    (2^-11 + e) A + 2^-32 N + 2^-8 |o|,    A = sum_j w_j |v_j|,  N = sum_j max(w) |v_j|,  e = D 2^-23 size + 2^-14,

the last term for o's one rounding to bf16; were P rounded to bf16, the first would be 2^-8. On the average over all
elements the roundings' signs are independent, 2^-11 sqrt(sum_j w_j^2 v_j^2), but for weights that are equal, which are
off alike: 2^-11 |o|. Rounding o is off by 2^-9 |o| on the average at most (a uniform error in half a step of 2^-8), and by a
quarter more where as few as 128 elements differ (five standard deviations). In all 2^-11 sqrt(..) + e A + 2^-32 N +
1.5 * 2^-9 |o|."""
import math

import numpy as np
import pytest
import torch

from oracle import paged as R
from tests import paged4_util as U
from tests import paged_util as P
from tests.paged_util import Batch

pytestmark = pytest.mark.gpu

SHAPES = [([1, 1], 8), ([4, 2], 4), ([4, 3], 8), ([5, 9], 8), ([16, 100], 1), ([150, 40], 8)]


def check(b, t, o, k_unit, v_unit, average=True):
    kp, vp = (U.values(t[x + "_pages"], t[x + "_scales"], u) for x, u in (("k", k_unit), ("v", v_unit)))
    table, q, got = t["table"].cpu().numpy(), t["q"].double().cpu().numpy(), o.double().cpu().numpy()
    off = allowed = 0.0
    row = 0
    for i, (n, length) in enumerate(zip(b.new, b.lens)):
        for h in range(b.hq):
            k, v = (P.sequence_rows(x, table, i, length, b.page, h * b.hkv // b.hq) for x in (kp, vp))
            ro, rl, spread, rms, size = R.attend(q[h, row:row + n], k, v, n, b.causal)
            for j in range(n):
                seen = length - n + j + 1 if b.causal else length
                s = k[:seen] @ q[h, row + j] / math.sqrt(b.d)
                largest = math.exp(s.max() - rl[j])
                small = 2.0 ** -32 * largest * np.abs(v[:seen]).sum(0) + 1e-30
                e = b.d * 2.0 ** -23 * size[j] + 2.0 ** -14
                err = np.abs(got[h, row + j] - ro[j])
                bound = (2.0 ** -11 + e) * spread[j] + small + 2.0 ** -8 * np.abs(ro[j])
                assert (err <= bound).all(), (i, h, j, float((err / bound).max()))
                off += err.sum()
                allowed += (2.0 ** -11 * rms[j] + e * spread[j] + small + 1.5 * 2.0 ** -9 * np.abs(ro[j])).sum()
        row += n
    assert off <= allowed or not average, (off, allowed)


def run(fcp, b, t, *units):
    cache, batch = U.handles(fcp, b, t, *units)
    o, _ = fcp.PagedAttention(cache, b.hq, causal=b.causal).forward(batch, t["q"])
    cache.check_device_error()
    return o


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,hq", SHAPES, ids=str)
def test_two_sets_of_keys_that_cancel(fcp, new, hq, d):
    """Every second key has the score S and V = 1, the others zero and V near -e^S: o is a few hundredths of the sums
    that it is the difference of, and the weights of the others are all rounded alike, so that rounding is its error."""
    b = Batch(new, [1000, 200], hq=hq, hkv=1, d=d, page=64, causal=False)
    for byte in (0x31, 0x33, 0x36, 0x39, 0x3B, 0x3D):  # the first keys' scale, from 0.56 to 1.6
        t = U.make(b)
        t["q"].fill_(0.125)
        score = math.sqrt(d) / 8 * float(R.e4m3_values()[byte])
        near = int(np.argmin(np.abs(R.e4m3_values()[:0x7F] - math.exp(score))))
        for x in "kv":
            t[x + "_pages"].view(torch.uint8).fill_(0x22)
            t[x + "_scales"].view(torch.uint8).fill_(byte if x == "k" else 0x38)
        t["k_pages"].view(torch.uint8)[:, :, 1::2] = 0
        t["v_pages"].view(torch.uint8)[:, :, 1::2] = 0xAA
        t["v_scales"].view(torch.uint8)[:, :, 1::2] = near
        check(b, t, run(fcp, b, t, 1.0, 1.0), 1.0, 1.0, average=False)  # the roundings are one and the same


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,hq", SHAPES, ids=str)
def test_many_small_weights_whose_sum_counts(fcp, new, hq, d):
    """One key with the score S and thousands at zero, e^-S of its weight each (2^-13 to 2^-24), whose values are 2^9 times
    the first's: without P's start at 2^7 they would be among f16's subnormal numbers or gone."""
    n = [4000, 3000]
    for power, at in ((13, 0), (15, 7), (18, 100), (21, 1500), (24, 2900)):
        b = Batch(new, n, hq=hq, hkv=1, d=d, page=64, causal=False)
        t = U.make(b)
        t["k_pages"].view(torch.uint8).zero_()
        # q is 2^-3 everywhere; a key of ones times a scale c has the score D c / 8 / sqrt(D)
        t["q"].fill_(0.125)
        want = power * math.log(2) * 8 / math.sqrt(d)
        scale = int(np.argmin(np.abs(R.e4m3_values()[:0x7F] - want)))
        t["v_scales"].view(torch.uint8).fill_(0x38 + 8 * 6)  # 2^6
        t["v_pages"].view(torch.uint8).copy_(torch.where(torch.rand(t["v_pages"].shape, device="cuda") < 0.75, 0x22, 0xAA))
        for i in range(2):
            page, row = int(t["table"][i, at // 64]), at % 64
            t["k_pages"].view(torch.uint8)[page, 0, row] = 0x22
            t["k_scales"].view(torch.uint8)[page, 0, row] = scale
            t["v_scales"].view(torch.uint8)[page, 0, row] = 0x38 - 8 * 3
        check(b, t, run(fcp, b, t, 1.0, 1.0), 1.0, 1.0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,hq", SHAPES, ids=str)
def test_scores_that_rise_along_the_keys(fcp, new, hq, d):
    """The running maximum is raised many times, by steps below and above what it lags behind, and sums of several groups
    of warps, pieces and blocks are joined."""
    b = Batch(new, [3000, 1200], hq=hq, hkv=1, d=d, page=32, causal=False)
    t = U.make(b)
    t["k_pages"].view(torch.uint8).fill_(0x22)
    t["q"] = (t["q"].abs() * 0.1 + 0.05).contiguous()
    for i, length in enumerate(b.lens):
        for pos in range(length):
            page, row = int(t["table"][i, pos // 32]), pos % 32
            t["k_scales"].view(torch.uint8)[page, 0, row] = 0x08 + (pos * 0x30) // length
    check(b, t, run(fcp, b, t, 16.0, 1.0), 16.0, 1.0)
