"""Attention over a 4-bit cache where q and the cache's unit are as large as they may be: the factor of the scores
is past float32's range, scores of zero are zero all the same."""
import pytest
import torch

from tests import paged4_util as U
from tests.paged_util import Batch

pytestmark = pytest.mark.gpu

SHAPES = [([1, 1], 4), ([3, 3], 4), ([3, 3], 16), ([5, 5], 8), ([50, 17], 4), ([200, 30], 4)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("unit,q", [(2.0 ** 60, 2.0 ** 100), (2.0 ** 60, 2.0 ** 126), (2.0 ** 20, 2.0 ** 127), (2.0 ** 60, 1.0)], ids=str)
@pytest.mark.parametrize("new,hq", SHAPES, ids=str)
def test_keys_of_zeros_weigh_the_same(fcp, new, hq, unit, q, d):
    """Every score is zero: o is the mean of V over the keys that a row sees, lse the logarithm of their number."""
    b = Batch(new, [300, 2 * new[1]], hq=hq, hkv=1, d=d, page=32, seed=len(new))
    t = U.make(b)
    t["k_pages"].view(torch.uint8).zero_()
    t["q"] = (t["q"].clamp(-1, 1) * q).contiguous()  # finite: 2^127 is the largest power of two
    cache, batch = U.handles(fcp, b, t, unit, 1.0)
    att = fcp.PagedAttention(cache, b.hq)
    o, lse = att.forward(batch, t["q"])
    cache.check_device_error()
    U.check_attention(b, {**t, "q": torch.zeros_like(t["q"])}, o, lse, k_unit=1.0, v_unit=1.0)


@pytest.mark.parametrize("new,hq", SHAPES, ids=str)
def test_one_key_that_is_not_zero(fcp, new, hq):
    """The only score that is not zero is far above or below the others: a row whose q agrees with the key has
    its V, one whose q does not has the mean of the others'. (Scores to 2^120, which float32 holds.)"""
    d, n = 64, 200
    b = Batch([new[0]], [n], hq=hq, hkv=1, d=d, page=32, causal=False)
    t = U.make(b)
    codes = t["k_pages"].view(torch.uint8)
    codes.zero_()
    page, row = int(t["table"][0, 100 // 32]), 100 % 32
    codes[page, 0, row, :] = 0x22  # 1.0 everywhere
    t["k_scales"].view(torch.uint8)[page, 0, row] = 0x38  # times 1
    t["q"].fill_(2.0 ** 57)
    t["q"][1::2] *= -1
    cache, batch = U.handles(fcp, b, t, 2.0 ** 60, 1.0)
    o, lse = fcp.PagedAttention(cache, b.hq, causal=False).forward(batch, t["q"])
    cache.check_device_error()
    v = torch.from_numpy(U.values(t["v_pages"], t["v_scales"], 1.0))
    v = torch.stack([v[int(t["table"][0, x // 32]), 0, x % 32] for x in range(n)])
    up, down = v[100], (v.sum(0) - v[100]) / (n - 1)
    spread = (v.abs().sum(0) - v[100].abs()) / (n - 1)
    o = o.double().cpu()
    # P's and o's roundings, as in paged_util
    assert ((o[0::2] - up).abs() <= (2.0 ** -7 + 2.0 ** -12) * up.abs()).all()
    assert ((o[1::2] - down).abs() <= 2.0 ** -8 * (spread + down.abs()) + 2.0 ** -12 * spread).all()
    score = 2.0 ** 57 * 2.0 ** 60 * d / 8.0
    assert ((lse[0::2].double().cpu() - score).abs() <= 2.0 ** -17 * score).all()
    assert ((lse[1::2].double().cpu() - torch.tensor(float(n - 1)).log().double()).abs() <= 1e-5).all()
