// Shared host/device definitions of the paged key/value cache: argument checks, the e8m0,
// e4m3 and e2m1 conversions, and a sequence's place in a batch.
//
// A cache row is one (token, KV head): D channels of K or of V. Rows live in pages
// [n_pages, Hkv, page_size, D], so the rows of one page and head are contiguous. In an e4m3
// cache a row carries a power-of-two scale 2^k kept as the byte k + 127 (e8m0; 255 is NaN):
// scaling by it is exact, so a row is rounded once when it is written and never again. A 4-bit cache
// has an e4m3 scale s for each 16 channels and a power of two for the whole cache: a code has 2
// significant bits and s has 4, so code * s is exact in f16 (at most 2688, multiples of 2^-10) and bf16.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <utility>

#include "fcp_cuda_util.h"
#include "fcp_sm100.cuh"

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
  float k_unit, v_unit;  // of a 4-bit cache; 1 otherwise
};

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

fcp_status paged_args(const fcp_cache* cache, const fcp_cache_batch* batch, PagedArgs* out);

// The cache's kernels are launched so that they may start while the kernel before them in the
// stream still runs, to hide the launch: each waits for that one's end before it touches
// memory, and lets the next one start in the same way.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Such a kernel is resident while what it reads may still be written, so nothing is read through
// the path for memory that stays the same as long as a kernel lives; and these loads keep their
// place behind the wait.
__device__ __forceinline__ int load(const int32_t* p) {
  int x;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(x) : "l"(p));
  return x;
}
__device__ __forceinline__ uint32_t load(const uint8_t* p) {
  uint32_t x;
  asm volatile("ld.global.u8 %0, [%1];" : "=r"(x) : "l"(p));
  return x;
}
__device__ __forceinline__ uint32_t load(const uint16_t* p) {
  uint32_t x;
  asm volatile("{\n.reg .b16 h;\nld.global.b16 h, [%1];\ncvt.u32.u16 %0, h;\n}" : "=r"(x) : "l"(p));
  return x;
}
__device__ __forceinline__ uint2 load(const uint2* p) {
  uint2 x;
  asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "l"(p));
  return x;
}
__device__ __forceinline__ uint4 load(const uint4* p) {
  uint4 x;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(p));
  return x;
}

template <int kCluster = 1, class... Params, class... Args>
inline fcp_status launch_overlapped(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t s,
                                    const char* where, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = kCluster > 1 ? 2 : 1;
  FCP_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...), where);
  return FCP_OK;
}

// The current device and its number of SMs, which does not change.
inline fcp_status this_device(int* dev, int* n_sm) {
  static std::atomic<int> known[64];
  FCP_CUDA_TRY(cudaGetDevice(dev), "paged cache device");
  if (*dev < 0 || *dev >= 64) return FCP_ERR_UNSUPPORTED;
  *n_sm = known[*dev].load(std::memory_order_relaxed);
  if (*n_sm == 0) {
    FCP_CUDA_TRY(cudaDeviceGetAttribute(n_sm, cudaDevAttrMultiProcessorCount, *dev), "paged cache SM count");
    known[*dev].store(*n_sm, std::memory_order_relaxed);
  }
  return FCP_OK;
}

// cudaFuncSetAttribute for a kernel's dynamic shared memory, once for each device.
template <class Kernel>
inline fcp_status allow_smem(Kernel kernel, int bytes, int device, std::atomic<uint64_t>& done, const char* where) {
  const uint64_t bit = 1ull << (device & 63);
  if (done.load(std::memory_order_relaxed) & bit) return FCP_OK;
  FCP_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes), where);
  done.fetch_or(bit, std::memory_order_relaxed);
  return FCP_OK;
}

// The rows [a, a + n) of sequence i and its cached length; n = 0 (with the error recorded by
// the thread that passes report) where they do not fit the batch.
struct SeqShape {
  int32_t a, n, len;
};
__device__ __forceinline__ SeqShape checked_shape(const PagedArgs& p, int a, int b, int len, bool report) {
  const bool ok = a >= 0 && b >= a && b <= p.total_new && len >= 0 &&
                  len <= (static_cast<long long>(p.max_pages) << p.page_shift);
  if (!ok && report) atomicCAS(p.status, 0, kErrCacheBatch);
  return SeqShape{a, ok ? b - a : 0, ok ? len : 0};
}
__device__ __forceinline__ SeqShape seq_shape(const PagedArgs& p, int i, bool report) {
  return checked_shape(p, load(p.cu + i), load(p.cu + i + 1), load(p.lens + i), report);
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

// Four e4m3 codes as two f16x2, exactly (the NaN codes as NaN).
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.rn.f16x2.e4m3x2 %0, a;\ncvt.rn.f16x2.e4m3x2 %1, b;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}

// Eight e2m1 codes as four f16x2 of neighbouring codes, exactly.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t eight, uint32_t (&r)[4]) {
  asm("{\n.reg .b8 a, b, c, d;\nmov.b32 {a, b, c, d}, %4;\ncvt.rn.f16x2.e2m1x2 %0, a;\ncvt.rn.f16x2.e2m1x2 %1, b;\n"
      "cvt.rn.f16x2.e2m1x2 %2, c;\ncvt.rn.f16x2.e2m1x2 %3, d;\n}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(eight));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t x, uint32_t y) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// An e4m3 scale as float32.
__device__ __forceinline__ float e4m3_to_float(uint32_t byte) {
  uint32_t lo, hi;
  e4m3x4_to_f16x2(byte, lo, hi);
  return __low2float(*reinterpret_cast<const __half2*>(&lo));
}

// 8 codes times their row's scale as 8 bf16 channels: the product with a power of two is exact in
// float32, and exact in bf16 while it is a normal number there.
__device__ __forceinline__ uint4 scaled8(const uint2 x, float scale) {
  uint32_t h[4], r[4];
  e4m3x4_to_f16x2(x.x, h[0], h[1]);
  e4m3x4_to_f16x2(x.y, h[2], h[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    const float2 y = dev::fmul2(v.x, v.y, scale, scale);
    r[i] = dev::pack_bf16(y.x, y.y);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// 8 e2m1 codes times a factor (a scale and the cache's unit) as 8 bf16 channels: exact as above.
__device__ __forceinline__ uint4 scaled8(uint32_t codes, float factor) {
  uint32_t h[4], r[4];
  e2m1x8_to_f16x2(codes, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    const float2 y = dev::fmul2(v.x, v.y, factor, factor);
    r[i] = dev::pack_bf16(y.x, y.y);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

}  // namespace fcp
