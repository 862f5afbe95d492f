"""The paged cache where its inputs are far from ordinary."""
import pytest
import torch

from tests import paged_util as U
from tests.paged_util import Batch
from tests.test_gpu_paged import attend

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- NaN in V
NAN_V = [
    # position, batch (sequence 0 holds the NaN)
    (94, Batch([10, 10], [100, 100], hq=2, hkv=1)),                        # among the new tokens, few rows each
    (96, Batch([6, 1], [100, 40], hq=8, hkv=2, d=128, page=32)),
    (85, Batch([40, 40], [100, 100], hq=2, hkv=1)),                        # chunks
    (290, Batch([200, 33], [300, 290], hq=8, hkv=2, d=128, page=64)),      # several tiles and units
    (3, Batch([100, 100], [100, 100], hq=4, hkv=1, d=128)),
    (5960, Batch([70, 5], [6000, 300], hq=4, hkv=1, page=128)),            # keys split over many blocks
    (200, Batch([70, 90], [6000, 300], hq=4, hkv=1, d=128, page=128)),     # seen by every row, in another block
    (250, Batch([60, 60], [300, 300], hq=2, hkv=1, causal=False)),
    (127, Batch([50, 3], [160, 3], hq=2, hkv=1, max_new=1)),               # the other kernel than the batch asks for
    (0, Batch([2, 3], [2, 3], hq=2, hkv=1, max_new=90)),
]


@pytest.mark.parametrize("c", ["bf16", "e4m3"])
@pytest.mark.parametrize("at,b", NAN_V, ids=lambda x: str(x))
def test_a_nan_in_v_reaches_its_readers(fcp, at, b, c):
    """A NaN row of V makes o of every row that sees it NaN and leaves lse as it is. Other sequences keep
    every bit, and in an e4m3 cache so do the rows that do not see it, whichever kernel runs."""
    b = Batch(**{**b.__dict__, "cache": c, "seed": at})
    t = U.make(b)
    cache, batch = U.handles(fcp, b, t)
    want = attend(fcp, b, t, cache, batch)
    for p in {at, max(at - 1, 0)}:  # one bad row, then two beside one another
        page, off = int(t["table"][0, p // b.page]), p % b.page
        if c == "bf16":
            t["v_pages"][page, :, off, 7] = float("nan")
        else:
            t["v_scales"].view(torch.uint8)[page, :, off] = 255
    first = max(at - 1, 0)
    o, lse, _ = attend(fcp, b, t, cache, batch)
    cache.check_device_error()
    n, length = b.new[0], b.lens[0]
    sees = (torch.arange(n) + length - n >= first).cuda() if b.causal else torch.ones(n, dtype=torch.bool, device="cuda")
    assert torch.equal(lse, want[1])
    assert torch.equal(o[:, n:], want[0][:, n:])
    if c == "bf16":  # rows before it: documented as not kept apart; other channels are not touched
        assert o[:, :n, 7][:, sees].isnan().all()
        keep = torch.arange(b.d, device="cuda") != 7
        assert torch.equal(o[:, :n][..., keep], want[0][:, :n][..., keep])
    else:
        assert o[:, :n][:, sees].isnan().all()
        assert torch.equal(o[:, :n][:, ~sees], want[0][:, :n][:, ~sees])


# ---------------------------------------------------------------- V's scales far apart
@pytest.mark.parametrize("new", [1, 2, 3, 8, 50], ids=lambda n: f"new{n}")
@pytest.mark.parametrize("apart", [6, 11, 18, 24, 40, 90])
@pytest.mark.parametrize("d", [64, 128])
def test_small_rows_of_v_beside_large_ones(fcp, new, apart, d):
    """Every ninth row of V is 2^apart larger than the rest, and zero but for one channel: the other
    channels are sums over the small rows alone, which must not be lost beside it."""
    b = Batch([new, 1], [300, 77], hq=4, hkv=1, d=d, page=32, cache="e4m3", seed=apart)
    t = U.make(b)
    codes, byte = t["v_pages"].view(torch.uint8), t["v_scales"].view(torch.uint8)
    large = torch.zeros_like(byte, dtype=torch.bool)
    large[:, :, 4::9] = True
    large &= byte != 255
    byte.copy_(torch.where(large, 117 + apart // 2, torch.where(byte == 255, 255, byte - (apart + 1) // 2)).to(torch.uint8))
    codes.masked_fill_(large[..., None] & (torch.arange(d, device="cuda") != 5), 0)
    cache, batch = U.handles(fcp, b, t)
    o, lse, before = attend(fcp, b, t, cache, batch)
    cache.check_device_error()
    U.check_attention(b, t, o, lse, *before)
