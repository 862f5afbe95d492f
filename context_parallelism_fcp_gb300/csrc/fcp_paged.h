// Shared host/device definitions of the paged key/value cache: argument checks, the e8m0 and
// e4m3 conversions, and a sequence's place in a batch.
//
// A cache row is one (token, KV head): D channels of K or of V. Rows live in pages
// [n_pages, Hkv, page_size, D], so the rows of one page and head are contiguous. In an e4m3
// cache a row carries a power-of-two scale 2^k kept as the byte k + 127 (e8m0; 255 is NaN):
// scaling by it is exact, so a row is rounded once when it is written and never again.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <utility>

#include "fcp_cuda_util.h"

namespace fcp {

// Device error codes of the cache calls (fcp_cache.status).
enum CacheError : int32_t {
  kErrCacheBatch = 0x50,  // a sequence's row offsets or length do not fit the batch
  kErrCachePage = 0x51,   // a block-table entry that is needed is outside [0, n_pages)
  kErrPagedWait = 0x60,   // .. 0x6f: a bounded wait of the chunk kernel gave up
};

// What the kernels need of fcp_cache and fcp_cache_batch.
struct PagedArgs {
  const int32_t* cu;
  const int32_t* lens;
  const int32_t* table;
  int32_t n_seqs, max_pages, n_pages, hkv;
  int32_t page_shift;
  int32_t total_new;
  uint8_t* k_pages;
  uint8_t* v_pages;
  uint8_t* k_scales;
  uint8_t* v_scales;
  int32_t* status;
};

fcp_status paged_args(const fcp_cache* cache, const fcp_cache_batch* batch, PagedArgs* out);

// The cache's kernels are launched so that they may start while the kernel before them in the
// stream still runs, to hide the launch: each waits for that one's end before it touches
// memory, and lets the next one start in the same way.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <class... Params, class... Args>
inline fcp_status launch_overlapped(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t s,
                                    const char* where, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  FCP_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...), where);
  return FCP_OK;
}

// The rows [a, a + n) of sequence i and its cached length; n = 0 (with the error recorded by
// the thread that passes report) where they do not fit the batch.
struct SeqShape {
  int32_t a, n, len;
};
__device__ __forceinline__ SeqShape seq_shape(const PagedArgs& p, int i, bool report) {
  const int a = __ldg(p.cu + i), b = __ldg(p.cu + i + 1), len = __ldg(p.lens + i);
  const bool ok = a >= 0 && b >= a && b <= p.total_new && len >= 0 &&
                  len <= (static_cast<long long>(p.max_pages) << p.page_shift);
  if (!ok && report) atomicCAS(p.status, 0, kErrCacheBatch);
  return SeqShape{a, ok ? b - a : 0, ok ? len : 0};
}

// First row of page `page` for head h (a row index into the pages and scales).
__device__ __forceinline__ long long page_row(const PagedArgs& p, int page, int h) {
  return (static_cast<long long>(page) * p.hkv + h) << p.page_shift;
}

// The scale 2^(b - 127) that byte b stands for, as float32 bits (b = 0 is 2^-127, 255 NaN).
__device__ __forceinline__ float e8m0_to_float(uint32_t b) {
  const uint32_t bits = b == 0u ? 0x00400000u : (b == 255u ? 0x7fc00000u : b << 23);
  return __uint_as_float(bits);
}

// log2 of the same.
__device__ __forceinline__ float e8m0_log2(uint32_t b) {
  return b == 255u ? __uint_as_float(0x7fc00000u) : static_cast<float>(static_cast<int>(b) - 127);
}

// Two e4m3 codes in bits 8-15 and 24-31 as bf16x2. The code's exponent and mantissa sit in
// bf16's fields with its bias 7 instead of 127, so one exact product with 2^120 gives the
// value; code subnormals are bf16 subnormals before it. (Codes 0x7f and 0xff, which a written
// cache never holds, read as +-480.)
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t x) {
  const uint32_t r = (x & 0x80008000u) | ((x & 0x7f007f00u) >> 4);
  const uint32_t f = 0x7b807b80u;  // 2^120
  __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&r), *reinterpret_cast<const __nv_bfloat162*>(&f));
  return *reinterpret_cast<uint32_t*>(&y);
}

}  // namespace fcp
