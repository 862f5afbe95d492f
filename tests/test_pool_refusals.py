"""The page pool's checks of its arguments, with no GPU (no call gets as far as a launch)."""
import ctypes

import pytest
import torch

INVALID, UNSUPPORTED = 1, 3
P = 1 << 12  # an aligned address that is never looked at


def _pool(**change):
    from context_parallelism_fcp_gb300 import _PagePoolStruct

    return _PagePoolStruct(**{**dict(free_pages=P, n_free=P, lens=P, block_table=P, status=P, n_pages=4, page_size=16,
                                     n_seqs=2, max_pages=3), **change})


@pytest.mark.parametrize("change,status", [
    (dict(n_pages=-1), INVALID), (dict(page_size=0), INVALID), (dict(n_seqs=-1), INVALID), (dict(max_pages=-1), INVALID),
    (dict(free_pages=None), INVALID), (dict(n_free=None), INVALID), (dict(lens=None), INVALID),
    (dict(block_table=None), INVALID), (dict(status=None), INVALID), (dict(status=P + 4), INVALID),
    (dict(lens=P + 2), INVALID), (dict(n_free=P + 1), INVALID), (dict(free_pages=P + 3), INVALID),
    (dict(block_table=P + 2), INVALID), (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED),
    (dict(page_size=8192), UNSUPPORTED), (dict(n_seqs=65537), UNSUPPORTED),
    (dict(page_size=4096, max_pages=(1 << 18) + 1), UNSUPPORTED)], ids=str)
def test_both_calls_refuse(fcp, change, status):
    L = fcp.lib()
    p = ctypes.byref(_pool(**change))
    assert L.fcp_pool_release(p, P, None) == status
    assert L.fcp_pool_admit(p, P, 5, P, 2 * P, P, P, None) == status


def test_buffers(fcp):
    L = fcp.lib()
    p = ctypes.byref(_pool())
    assert L.fcp_pool_release(None, P, None) == INVALID and L.fcp_pool_release(p, None, None) == INVALID
    assert L.fcp_pool_release(p, P + 2, None) == INVALID
    good = [p, P, 5, P, 2 * P, P, P, None]
    for at, value, status in ((0, None, INVALID), (1, None, INVALID), (1, P + 1, INVALID), (2, -1, INVALID), (3, None, INVALID),
                              (3, P + 2, INVALID), (4, None, INVALID), (4, P + 2, INVALID), (4, P, INVALID), (5, P + 2, INVALID),
                              (6, P + 4, INVALID), (2, (1 << 30) + 1, UNSUPPORTED)):
        args = list(good)
        args[at] = value
        assert L.fcp_pool_admit(*args) == status, (at, value)
    assert L.fcp_pool_release(ctypes.byref(_pool(n_seqs=0, lens=None, block_table=None)), None, None) == 0


def test_the_binding_takes_cuda_tensors_only(fcp):
    ints = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fcp.PagePool.wrap(ints, ints[:1], ints, ints.view(2, 1), 16)
    with pytest.raises(ValueError, match="CUDA"):
        fcp.PagePool(4, 16, 2, 2, device="cpu")
    assert "PagePool" in fcp.__all__
