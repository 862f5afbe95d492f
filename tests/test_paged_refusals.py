"""The paged cache's checks of its arguments: status codes of the C calls and errors of the binding,
with no GPU (no call gets as far as a launch)."""
import ctypes

import pytest
import torch

INVALID, UNSUPPORTED = 1, 3
P = 1 << 12  # an aligned address that is never looked at


def _structs(fcp, **change):
    from context_parallelism_fcp_gb300 import _CacheBatchStruct, _CacheStruct

    cache = dict(k_pages=P, v_pages=P, k_scales=P, v_scales=P, status=P, n_pages=4, hkv=2, page_size=16, head_dim=64,
                 dtype=1, reserved=0)
    batch = dict(cu_new=P, lens=P, block_table=P, n_seqs=2, max_pages=3, total_new=5, max_new=4)
    for k, v in change.items():
        (cache if k in cache else batch)[k] = v
    return _CacheStruct(**cache), _CacheBatchStruct(**batch)


BAD = [
    (dict(n_pages=-1), INVALID), (dict(hkv=0), INVALID), (dict(page_size=0), INVALID), (dict(n_seqs=-1), INVALID),
    (dict(max_pages=-1), INVALID), (dict(total_new=-1), INVALID), (dict(max_new=-1), INVALID), (dict(dtype=2), INVALID),
    (dict(status=None), INVALID), (dict(status=P + 4), INVALID), (dict(k_pages=None), INVALID),
    (dict(v_pages=P + 8), INVALID), (dict(k_scales=None), INVALID), (dict(v_scales=P + 1), INVALID),
    (dict(cu_new=None), INVALID), (dict(lens=None), INVALID), (dict(block_table=None), INVALID),
    (dict(head_dim=96), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED),
    (dict(page_size=8192), UNSUPPORTED), (dict(n_seqs=65537), UNSUPPORTED),
    (dict(page_size=4096, max_pages=1 << 20), UNSUPPORTED), (dict(page_size=4096, max_pages=(1 << 18) + 1), UNSUPPORTED),
    (dict(total_new=(1 << 30) + 1), UNSUPPORTED), (dict(cu_new=P + 2), INVALID), (dict(lens=P + 1), INVALID), (dict(block_table=P + 3), INVALID),
]


@pytest.mark.parametrize("change,status", BAD, ids=lambda x: str(x))
def test_every_call_refuses(fcp, change, status):
    L = fcp.lib()
    c, b = (ctypes.byref(x) for x in _structs(fcp, **change))
    ws = L.fcp_paged_attn_workspace_bytes(64)
    assert L.fcp_cache_write(c, b, P, P, None) == status
    assert L.fcp_cache_read(c, b, P, P, None) == status
    assert L.fcp_paged_attn(c, b, P, 4, 1, P, P, P, ws, None) == status


def test_nulls_and_misaligned_buffers(fcp):
    L = fcp.lib()
    c, b = (ctypes.byref(x) for x in _structs(fcp))
    ws = L.fcp_paged_attn_workspace_bytes(64)
    assert ws > 0 and L.fcp_paged_attn_workspace_bytes(128) > ws and L.fcp_paged_attn_workspace_bytes(32) == 0
    for k, v in ((None, P), (P, None), (P + 2, P), (P, P + 8)):
        assert L.fcp_cache_write(c, b, k, v, None) == INVALID
        assert L.fcp_cache_read(c, b, k, v, None) == INVALID
    good = [c, b, P, 4, 1, P, P, P, ws, None]
    for at, value in ((0, None), (1, None), (2, None), (2, P + 8), (3, 0), (3, 3), (3, -2), (5, None), (5, P + 8),
                      (6, None), (6, P + 2), (7, None), (7, P + 16), (8, ws - 1)):
        args = list(good)
        args[at] = value
        assert L.fcp_paged_attn(*args) == INVALID, (at, value)
    assert L.fcp_cache_write(None, b, P, P, None) == INVALID and L.fcp_cache_read(c, None, P, P, None) == INVALID


def test_nothing_to_do_needs_no_buffers(fcp):
    L = fcp.lib()
    for change in (dict(total_new=0), dict(n_seqs=0, cu_new=None, lens=None, block_table=None)):
        c, b = (ctypes.byref(x) for x in _structs(fcp, **change))
        assert L.fcp_cache_write(c, b, None, None, None) == 0
        assert L.fcp_cache_read(c, b, None, None, None) == 0
        assert L.fcp_paged_attn(c, b, None, 2, 1, None, None, None, 0, None) == 0


def test_the_binding_takes_cuda_tensors_only(fcp):
    pages = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        fcp.PagedCache.wrap(pages, pages.clone())
    with pytest.raises(TypeError):
        fcp.PagedCache.wrap(pages.float(), pages.float())
    with pytest.raises(TypeError):
        fcp.PagedCache(2, 16, 1, 64, dtype=torch.float16, device="cpu")
    ints = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fcp.CacheBatch(ints, ints[:1], ints[:1].view(1, 1), 1, max_new=1)


def test_the_package_offers_the_cache_by_name(fcp):
    for name in ("PagedCache", "CacheBatch", "cache_write", "cache_read", "paged_attn", "PagedAttention"):
        assert name in fcp.__all__ and callable(getattr(fcp, name))
    with pytest.raises(AttributeError):
        fcp.no_such_name
