"""The 4-bit cache's checks of its arguments, with no GPU (no call gets as far as a launch), and its
oracle against what is known of it."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import paged4 as R4

INVALID = 1
P = 1 << 12  # an aligned address that is never looked at


def _structs(**change):
    from context_parallelism_fcp_gb300 import _CacheBatchStruct, _CacheStruct

    cache = dict(k_pages=P, v_pages=P, k_scales=P, v_scales=P, status=P, n_pages=4, hkv=2, page_size=16, head_dim=64,
                 dtype=2, reserved=0, k_unit=1.0, v_unit=0.5)
    cache.update(change)
    return _CacheStruct(**cache), _CacheBatchStruct(cu_new=P, lens=P, block_table=P, n_seqs=2, max_pages=3, total_new=5,
                                                    max_new=4)


@pytest.mark.parametrize("change", [dict(k_scales=None), dict(v_scales=P + 1), dict(k_pages=P + 8), dict(k_unit=0.0),
                                    dict(v_unit=-1.0), dict(k_unit=3.0), dict(v_unit=float("nan")), dict(dtype=3),
                                    dict(k_unit=float("inf")), dict(v_unit=2.0 ** 61), dict(k_unit=2.0 ** -61)], ids=str)
def test_every_call_refuses(fcp, change):
    L = fcp.lib()
    c, b = (ctypes.byref(x) for x in _structs(**change))
    assert L.fcp_cache_write(c, b, P, P, None) == INVALID
    assert L.fcp_cache_read(c, b, P, P, None) == INVALID
    assert L.fcp_paged_attn(c, b, P, 4, 1, P, P, P, L.fcp_paged_attn_workspace_bytes(64), None) == INVALID


def test_units_at_the_ends_of_their_range(fcp):
    from context_parallelism_fcp_gb300 import _CacheBatchStruct

    none = _CacheBatchStruct(cu_new=P, lens=P, block_table=P, n_seqs=0, max_pages=0, total_new=0, max_new=0)
    for u in (2.0 ** -60, 2.0 ** 60):
        c, _ = _structs(k_unit=u, v_unit=u)
        assert fcp.lib().fcp_cache_write(ctypes.byref(c), ctypes.byref(none), None, None, None) == 0


def test_the_binding_refuses(fcp):
    codes = torch.zeros(2, 1, 16, 32, dtype=torch.uint8)
    with pytest.raises(TypeError, match="float4_e2m1fn_x2"):
        fcp.PagedCache.wrap(codes, codes)
    with pytest.raises(ValueError, match="CUDA"):
        fcp.PagedCache.wrap(*(codes.view(torch.float4_e2m1fn_x2) for _ in "kv"))
    with pytest.raises(ValueError, match="head_dim"):
        fcp.PagedCache(2, 16, 1, 96, dtype=torch.float4_e2m1fn_x2, device="cpu")


def test_the_oracle(fcp):
    """Values that are known by hand: borders go to even codes, scales to even e4m3 codes, 6 is the most."""
    row = np.zeros(16)
    row[:9] = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.26]
    codes, scale = R4.quantise(row[None], 1.0)
    assert scale.tolist() == [[0x38]] and codes[0, :9].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 9]
    assert R4.value(codes, scale, 1.0)[0, :9].tolist() == [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, -0.5]
    # a sixth of the largest between two scales: 1.0625 is half-way from 1 to 1.125, and goes to 1
    row[0] = 6.375
    codes, scale = R4.quantise(row[None], 1.0)
    assert scale.tolist() == [[0x38]] and codes[0, 0] == 7
    assert R4.quantise(np.full((1, 16), 1e9), 4.0)[1].tolist() == [[0x7E]]
    assert R4.quantise(np.zeros((1, 16)), 1.0)[1].tolist() == [[1]]
    assert R4.unpack(np.array([[0x21, 0xF0]], np.uint8)).tolist() == [[1, 2, 0, 15]]
