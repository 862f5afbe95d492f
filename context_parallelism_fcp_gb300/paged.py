"""The paged key/value cache of include/fcp.h and the attention that reads it.

``PagedCache`` holds one layer's pages, ``CacheBatch`` says which rows of a packed batch belong
to which cached sequence, and ``cache_write``, ``cache_read`` and ``paged_attn`` are the C calls
of the same names. As in the rest of the package the arguments are checked and marshalled here
and all the work is done by the library's kernels, on the caller's stream. That may be any stream: what a
cache or an attention allocates stays theirs until the work of every stream that they were used on is done.
(Tensors of the caller's follow torch's rule: one that is used on another stream than its own and then dropped
is the caller's to record there. A graph's tensors and objects have to outlive it.)
"""
from __future__ import annotations

import ctypes
import sys
from contextlib import nullcontext
from typing import Optional, Tuple

import torch

from . import _CacheBatchStruct, _CacheStruct, _check, _need, _stream, device_error, FcpError, lib

__all__ = ["PagedCache", "CacheBatch", "cache_write", "cache_read", "paged_attn", "PagedAttention"]

_DTYPES = {torch.bfloat16: 0, torch.float8_e4m3fn: 1}


def _here(index: int, stream) -> int:
    """The stream to launch on. Kernels run on the current device, so that is where the tensors
    have to be."""
    if torch._C._cuda_getDevice() != index:
        raise ValueError(f"the cache is on cuda:{index}, the current device is cuda:{torch._C._cuda_getDevice()}")
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream(stream)


def _want(t, dtype, shape, index: int, name: str) -> None:
    """_need and the device, with a step's few microseconds in mind: what is right passes quickly."""
    if (type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape and t.get_device() == index
            and t.is_contiguous()):
        return
    _need(t, dtype, shape, name)
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the cache on cuda:{index}")


class _Owner:
    """An object with device memory of its own that calls on any stream may use. The allocator knows that
    memory as the stream's that was current when the object was made: so the object waits there until what
    that stream did with it before is done, and lets the allocator know of every other stream that uses it."""

    _foreign = False

    def _own(self, tensors, index: int) -> None:
        self._tensors, self._index = tensors, index
        self._streams = {torch._C._cuda_getCurrentRawStream(index)}
        with torch.cuda.device(index):
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()

    def _note(self, raw: int, stream) -> None:
        """Called for a stream that is not in _streams yet."""
        self._streams.add(raw)
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.current_stream(self._index) if stream is None else None
        if stream is None or (raw != 0 and stream.stream_id == raw):
            self._foreign = True  # made elsewhere, and perhaps destroyed before this object
            return
        for t in self._tensors:
            t.record_stream(stream)

    def __del__(self):
        if self._foreign and not sys.is_finalizing() and not torch.cuda.is_current_stream_capturing():
            torch.cuda.synchronize(self._index)


class PagedCache(_Owner):
    """K and V of one layer in pages (fcp_cache). ``dtype`` is torch.bfloat16, or
    torch.float8_e4m3fn for a cache that quantises each row as it is written, with a
    power-of-two scale for each token and head. Pages start as zeros."""

    def __init__(self, n_pages: int, page_size: int, hkv: int, head_dim: int, dtype=torch.bfloat16, device="cuda"):
        if dtype not in _DTYPES:
            raise TypeError(f"dtype must be torch.bfloat16 or torch.float8_e4m3fn, got {dtype}")
        shape = (int(n_pages), int(hkv), int(page_size), int(head_dim))
        pages = [torch.zeros(shape, dtype=torch.uint8 if dtype != torch.bfloat16 else dtype, device=device)
                 for _ in range(2)]
        scales = [None, None]
        if dtype != torch.bfloat16:
            pages = [p.view(dtype) for p in pages]
            scales = [torch.full(shape[:3], 127, dtype=torch.uint8, device=device).view(torch.float8_e8m0fnu)
                      for _ in range(2)]
        self._setup(*pages, *scales, made=[*pages, *(x for x in scales if x is not None)])

    @classmethod
    def wrap(cls, k_pages, v_pages, k_scales=None, v_scales=None) -> "PagedCache":
        """A cache over pages that exist already ([n_pages, Hkv, page_size, D], and for e4m3 pages
        the e8m0 scales [n_pages, Hkv, page_size])."""
        self = cls.__new__(cls)
        self._setup(k_pages, v_pages, k_scales, v_scales)
        return self

    def _setup(self, k_pages, v_pages, k_scales, v_scales, made=()):
        if not isinstance(k_pages, torch.Tensor) or k_pages.dtype not in _DTYPES:
            raise TypeError("k_pages must be a torch tensor of bfloat16 or float8_e4m3fn")
        if k_pages.dim() != 4:
            raise ValueError("k_pages must have shape [n_pages, Hkv, page_size, D]")
        if k_pages.shape[1] == 0:
            raise ValueError("k_pages must have a KV head at least")
        _need(k_pages, k_pages.dtype, None, "k_pages")
        _need(v_pages, k_pages.dtype, k_pages.shape, "v_pages")
        quantised = k_pages.dtype != torch.bfloat16
        for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
            if quantised:
                _need(t, torch.float8_e8m0fnu, k_pages.shape[:3], name)
            elif t is not None:
                raise ValueError(f"{name}: a bf16 cache has no scales")
        tensors = [t for t in (k_pages, v_pages, k_scales, v_scales) if t is not None]
        if any(t.device != k_pages.device for t in tensors):
            raise ValueError("the cache's tensors must be on one device")
        self.k_pages, self.v_pages, self.k_scales, self.v_scales = k_pages, v_pages, k_scales, v_scales
        self.n_pages, self.hkv, self.page_size, self.head_dim = (int(x) for x in k_pages.shape)
        if self.head_dim not in (64, 128):
            raise ValueError(f"head_dim must be 64 or 128, got {self.head_dim}")
        if self.page_size not in (16, 32, 64, 128, 256, 512, 1024, 2048, 4096):
            raise ValueError(f"page_size must be a power of two from 16 to 4096, got {self.page_size}")
        self.dtype, self.device = k_pages.dtype, k_pages.device
        self.status = torch.zeros(64, dtype=torch.int32, device=self.device)
        self._own([self.status, *made], k_pages.get_device())
        self._struct = _CacheStruct(
            k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr() if quantised else None,
            v_scales.data_ptr() if quantised else None, self.status.data_ptr(), self.n_pages, self.hkv,
            self.page_size, self.head_dim, _DTYPES[self.dtype], 0)
        self._ref = ctypes.byref(self._struct)

    def check_device_error(self, stream=None) -> None:
        """Synchronise and raise if a kernel recorded an error for this cache (see fcp_cache)."""
        code = device_error(self.status, stream)
        if code:
            raise FcpError(6, "paged cache", f"error word 0x{code:x}")


class CacheBatch:
    """The new tokens of a batch (fcp_cache_batch): sequence i owns packed rows [cu_new[i],
    cu_new[i+1]) of ``total_new`` and has ``lens[i]`` tokens in the cache, the new ones included;
    ``block_table[i]`` lists its pages. All three are int32 CUDA tensors that the kernels read when
    they run, so they can be updated in place between steps or replays. ``max_new``: the most new
    tokens of any sequence (it chooses the kernel and decides nothing else)."""

    def __init__(self, cu_new, lens, block_table, total_new: int, max_new: int):
        _need(lens, torch.int32, None, "lens")
        if lens.dim() != 1:
            raise ValueError("lens must have shape [n_seqs]")
        n = lens.shape[0]
        _need(cu_new, torch.int32, (n + 1,), "cu_new")
        _need(block_table, torch.int32, None, "block_table")
        if block_table.dim() != 2 or block_table.shape[0] != n:
            raise ValueError(f"block_table must have shape [{n}, max_pages], got {tuple(block_table.shape)}")
        if int(total_new) < 0 or int(max_new) < 0:
            raise ValueError("total_new and max_new must not be negative")
        if cu_new.device != lens.device or block_table.device != lens.device:
            raise ValueError("the batch's tensors must be on one device")
        self.cu_new, self.lens, self.block_table = cu_new, lens, block_table
        self.n_seqs, self.total_new, self.max_new, self.device = n, int(total_new), int(max_new), lens.device
        self._index = lens.get_device()
        self._struct = _CacheBatchStruct(cu_new.data_ptr(), lens.data_ptr(), block_table.data_ptr(), n,
                                         block_table.shape[1], self.total_new, self.max_new)
        self._ref = ctypes.byref(self._struct)


def _move(fn, name, cache: PagedCache, batch: CacheBatch, k, v, stream) -> None:
    index = cache._index
    if batch._index != index:
        raise ValueError("the batch and the cache must be on one device")
    shape = (cache.hkv, batch.total_new, cache.head_dim)
    _want(k, torch.bfloat16, shape, index, "k")
    _want(v, torch.bfloat16, shape, index, "v")
    raw = _here(index, stream)
    if raw not in cache._streams:
        cache._note(raw, stream)
    status = fn(cache._ref, batch._ref, k.data_ptr(), v.data_ptr(), raw)
    if status:
        _check(status, name)


def cache_write(cache: PagedCache, batch: CacheBatch, k, v, stream=None) -> None:
    """Write the new tokens' K and V (bf16 [Hkv, total_new, D]) into their pages, quantising them
    where the cache is e4m3 (fcp_cache_write)."""
    _move(lib().fcp_cache_write, "fcp_cache_write", cache, batch, k, v, stream)


def cache_read(cache: PagedCache, batch: CacheBatch, k, v, stream=None) -> None:
    """Read the batch's rows of the cache back into bf16 k and v [Hkv, total_new, D]
    (fcp_cache_read); rows that belong to no sequence are left as they were."""
    _move(lib().fcp_cache_read, "fcp_cache_read", cache, batch, k, v, stream)


def paged_attn(cache: PagedCache, batch: CacheBatch, q, o, lse, workspace, causal: bool = True, stream=None) -> None:
    """Attention of the new tokens' queries q [Hq, total_new, D] over their sequences' cached rows,
    into o (bf16, as q) and lse (float32 [Hq, total_new]) (fcp_paged_attn). The new tokens' K and V
    must be in the cache. workspace: a CUDA uint8 tensor of fcp_paged_attn_workspace_bytes(D)."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a tensor [Hq, total_new, D]")
    _need(workspace, torch.uint8, None, "workspace")
    if workspace.get_device() != cache._index:
        raise ValueError("the workspace and the cache must be on one device")
    _attend(lib().fcp_paged_attn, cache, batch, q, o, lse, workspace.data_ptr(), workspace.nbytes, 1 if causal else 0,
            q.shape[0], stream)


def _attend(fn, cache, batch, q, o, lse, workspace, workspace_bytes, causal, hq, stream, owner=None) -> None:
    index = cache._index
    if batch._index != index:
        raise ValueError("the batch and the cache must be on one device")
    shape = (hq, batch.total_new, cache.head_dim)
    _want(q, torch.bfloat16, shape, index, "q")
    _want(o, torch.bfloat16, shape, index, "o")
    _want(lse, torch.float32, shape[:2], index, "lse")
    raw = _here(index, stream)
    if raw not in cache._streams:
        cache._note(raw, stream)
    if owner is not None and raw not in owner._streams:
        owner._note(raw, stream)
    status = fn(cache._ref, batch._ref, q.data_ptr(), hq, causal, o.data_ptr(), lse.data_ptr(), workspace,
                workspace_bytes, raw)
    if status:
        _check(status, "fcp_paged_attn")


class PagedAttention(_Owner):
    """paged_attn with a workspace of its own, for one cache. Calls that may overlap on the GPU
    (other streams, replays of captured graphs) need one PagedAttention each."""

    def __init__(self, cache: PagedCache, hq: int, causal: bool = True):
        if hq <= 0 or hq % cache.hkv != 0:
            raise ValueError(f"hq must be a multiple of the cache's {cache.hkv} KV heads, got {hq}")
        self.cache, self.hq, self.causal = cache, int(hq), bool(causal)
        self.workspace = torch.empty(int(lib().fcp_paged_attn_workspace_bytes(cache.head_dim)), dtype=torch.uint8,
                                     device=cache.device)
        self._own([self.workspace], cache._index)
        self._call = lib().fcp_paged_attn, cache
        self._last = self.workspace.data_ptr(), self.workspace.nbytes, 1 if causal else 0, self.hq

    def forward(self, batch: CacheBatch, q, o=None, lse=None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        """(o, lse) of the batch's new tokens; rows that belong to no sequence are left as they
        were in the buffers given, and are undefined in those that are allocated here (as memory
        of the stream that the call runs on)."""
        if o is None or lse is None:
            if stream is not None and not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(_stream(stream), device=q.device)
            with nullcontext() if stream is None else torch.cuda.stream(stream):
                o = torch.empty_like(q) if o is None else o
                lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device) if lse is None else lse
        _attend(*self._call, batch, q, o, lse, *self._last, stream, self)
        return o, lse
