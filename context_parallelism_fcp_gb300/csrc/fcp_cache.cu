// Writing rows of K and V into the pages of a paged cache (quantising them where the cache is
// e4m3), and reading them back as bf16.
//
// Row r = (token, KV head) with channels x: an e4m3 cache stores k = the smallest integer
// >= -126 with max|x| <= 448 * 2^k, and the codes e4m3(x * 2^-k), rounded to nearest even: the
// only rounding there is, since the product with a power of two is exact. Reading gives
// code * 2^k, exact in bf16 (a code has 4 significant bits) while it is a normal number. A row
// with an infinity or NaN in it gets the NaN scale and zero codes: it reads back as NaN.
//
// Both directions are bound by HBM: 2 * T * Hkv rows in and out, nothing reused. A warp moves whole
// rows, D / 8 lanes to a row, 16 bytes of bf16 to a lane; a block takes 32 tokens of all heads, whose
// places are looked up once. Measured, D = 128: 27000 new tokens of 8 heads written into an e4m3
// cache in 32.2 us (5220 GB/s, 77% of a copy's rate; the third round of blocks is a quarter full),
// 169000 of 4 heads in 90 us (5780 GB/s), 35000 tokens of 8 heads read in 37 us (5800 GB/s); bf16
// caches 6300 (write) to 7000 GB/s (read).
// Writing e4m3 was bound by integer instructions (33.3 and 101 us) until pointers stepped along and
// the clamp of the largest scale became a branch of its own.
#include <algorithm>
#include <type_traits>

#include "fcp_paged.h"

namespace fcp {

fcp_status paged_args(const fcp_cache* c, const fcp_cache_batch* b, PagedArgs* out) {
  if (c == nullptr || b == nullptr || out == nullptr) return FCP_ERR_INVALID;
  if (c->n_pages < 0 || c->hkv <= 0 || c->page_size <= 0 || b->n_seqs < 0 || b->max_pages < 0 || b->total_new < 0 ||
      b->max_new < 0)
    return FCP_ERR_INVALID;
  if (c->dtype != FCP_CACHE_BF16 && c->dtype != FCP_CACHE_E4M3) return FCP_ERR_INVALID;
  if (c->head_dim != 64 && c->head_dim != 128) return FCP_ERR_UNSUPPORTED;
  if (c->page_size < 16 || c->page_size > 4096 || (c->page_size & (c->page_size - 1)) != 0) return FCP_ERR_UNSUPPORTED;
  if (static_cast<long long>(b->max_pages) * c->page_size > 1ll << 30) return FCP_ERR_UNSUPPORTED;
  if (b->n_seqs > 65536 || b->total_new > 1 << 30) return FCP_ERR_UNSUPPORTED;
  if (c->status == nullptr || !aligned16(c->status)) return FCP_ERR_INVALID;
  if (b->n_seqs > 0 && (!b->cu_new || !b->lens || (b->max_pages > 0 && !b->block_table))) return FCP_ERR_INVALID;
  if (!aligned4(b->cu_new) || !aligned4(b->lens) || !aligned4(b->block_table)) return FCP_ERR_INVALID;
  if (c->n_pages > 0) {
    if (!c->k_pages || !c->v_pages || !aligned16(c->k_pages) || !aligned16(c->v_pages)) return FCP_ERR_INVALID;
    if (c->dtype == FCP_CACHE_E4M3 &&
        (!c->k_scales || !c->v_scales || !aligned16(c->k_scales) || !aligned16(c->v_scales)))
      return FCP_ERR_INVALID;
  }
  PagedArgs p;
  p.cu = b->cu_new;
  p.lens = b->lens;
  p.table = b->block_table;
  p.n_seqs = b->n_seqs;
  p.max_pages = b->max_pages;
  p.n_pages = c->n_pages;
  p.hkv = c->hkv;
  p.page_shift = 0;
  while ((1 << p.page_shift) < c->page_size) ++p.page_shift;
  p.total_new = b->total_new;
  p.k_pages = static_cast<uint8_t*>(c->k_pages);
  p.v_pages = static_cast<uint8_t*>(c->v_pages);
  p.k_scales = c->k_scales;
  p.v_scales = c->v_scales;
  p.status = c->status;
  if (c->n_pages == 0) p.k_pages = p.v_pages = p.k_scales = p.v_scales = reinterpret_cast<uint8_t*>(c->status);
  *out = p;
  return FCP_OK;
}

namespace {

constexpr int kMoveThreads = 256;
constexpr int kMoveTokens = 32;   // packed rows of a block
constexpr int kCoarse = 1024;     // row offsets kept in shared memory
constexpr int kEnough = 8;        // blocks of an SM: all that its threads allow

// The cache row (page * page_size + offset, to which a head adds its stride) of each of the
// block's tokens; -1 for rows behind the last sequence, rows before their sequence's first
// position and rows whose page is outside the cache.
struct TokenPlace {
  int32_t page, off;
};

__device__ __forceinline__ void find_places(const PagedArgs& p, int t0, TokenPlace* place, int* coarse, int* lens) {
  // The last i with cu[i] <= t: every `step`-th offset is searched in shared memory and the
  // rest in memory, so that the dependent reads are few however many sequences there are. Where
  // step is 1 the lengths come with the offsets, and the page is the only dependent read.
  const int step = (p.n_seqs + kCoarse) / kCoarse;
  const int n_coarse = (p.n_seqs + step) / step;  // offsets 0, step, ... <= n_seqs
  for (int j = threadIdx.x; j < n_coarse; j += kMoveThreads) {
    coarse[j] = load(p.cu + j * step);
    if (step == 1 && j < p.n_seqs) lens[j] = load(p.lens + j);
  }
  __syncthreads();
  const int t = t0 + threadIdx.x;
  const bool mine = threadIdx.x < kMoveTokens && t < p.total_new;
  int i = 0;
  SeqShape s{0, 0, 0};
  if (mine) {
    int lo = 0, hi = n_coarse;  // coarse[lo] <= t < coarse[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (coarse[mid] <= t) lo = mid; else hi = mid;
    }
    i = lo * step;
    int e = min(i + step, p.n_seqs);
    while (e - i > 1) {
      const int mid = (i + e) >> 1;
      if (load(p.cu + mid) <= t) i = mid; else e = mid;
    }
    if (i < p.n_seqs) s = step == 1 ? checked_shape(p, coarse[i], coarse[i + 1], lens[i], true) : seq_shape(p, i, true);
  }
  const bool lost = mine && (s.n == 0 || t < s.a || t >= s.a + s.n);
  if (__syncthreads_or(lost)) {
    // Rows before the first sequence and behind the last, but also rows of a batch whose offsets fall
    // back, in which the search may miss the sequence that owns one: every sequence is asked.
    int* owner = reinterpret_cast<int*>(place);
    if (threadIdx.x < kMoveTokens) owner[threadIdx.x] = -1;
    __syncthreads();
    for (int base = 0; base < p.n_seqs; base += kCoarse - 1) {
      if (step > 1) {
        __syncthreads();
        for (int j = threadIdx.x; j < kCoarse; j += kMoveThreads) coarse[j] = load(p.cu + min(base + j, p.n_seqs));
        __syncthreads();
      }
      for (int j = threadIdx.x; j < min(kCoarse - 1, p.n_seqs - base); j += kMoveThreads) {
        if (coarse[j] >= t0 + kMoveTokens || coarse[j + 1] <= t0) continue;
        const SeqShape z = seq_shape(p, base + j, false);
        if (z.n > 0)
          for (int x = max(z.a - t0, 0); x < min(z.a + z.n - t0, kMoveTokens); ++x) atomicMax(&owner[x], base + j);
      }
    }
    __syncthreads();
    if (lost) {
      i = owner[threadIdx.x];
      s = i >= 0 ? seq_shape(p, i, false) : SeqShape{0, 0, 0};
    }
    __syncthreads();
  }
  if (threadIdx.x < kMoveTokens) {
    TokenPlace r{-1, 0};
    const int pos = s.n > 0 ? s.len - s.n + (t - s.a) : -1;
    if (pos >= 0) {
      const int page = load(p.table + static_cast<long long>(i) * p.max_pages + (pos >> p.page_shift));
      if (page >= 0 && page < p.n_pages) {
        r.page = page;
        r.off = pos & ((1 << p.page_shift) - 1);
      } else {
        atomicCAS(p.status, 0, kErrCachePage);
      }
    }
    place[threadIdx.x] = r;
  }
  __syncthreads();
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t min_u16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("min.u16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// Quantise the 8 channels of this lane (of a row shared by LPR lanes): 8 codes and the row's scale byte.
template <int LPR>
__device__ __forceinline__ uint2 quantise(const uint4 x, uint32_t& scale_byte) {
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
  // the largest magnitude as bf16 bits, two channels at a time: non-finite values order above
  // every finite one
  uint32_t two = max_u16x2(max_u16x2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu), max_u16x2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) two = max_u16x2(two, __shfl_xor_sync(0xffffffffu, two, o));
  const uint32_t top = max(two & 0xffffu, two >> 16);
  // max|x| = 1.m * 2^e <= 1.75 * 2^(8 + k): k = e - 8, or e - 7 where 1.m > 1.75 (mantissa over 0x60,
  // which carries into the exponent here)
  uint32_t byte = top == 0u ? 127u : static_cast<uint32_t>(max(static_cast<int>((top + 0x1fu) >> 7) - 8, 1));
  if (__any_sync(0xffffffffu, top > 0x7f60u)) {
    // k = 120: 256 * 2^120 is the one product that bf16 cannot hold; or an infinity or NaN
    if (top > 0x7f60u) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = top >= 0x7f80u ? 0u : (w[i] & 0x80008000u) | min_u16x2(w[i] & 0x7fff7fffu, 0x7f707f70u);
      if (top >= 0x7f80u) byte = 255u;
    }
  }
  scale_byte = byte;
  const float inv = __uint_as_float((254u - min(byte, 253u)) << 23);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = __nv_cvt_float2_to_fp8x2(dev::fmul2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u), inv, inv),
                                    __NV_SATFINITE, __NV_E4M3);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// grid (ceil(T / 32), ceil(Hkv / heads per block), 2: K or V)
template <int D, bool kE4M3, bool kRead>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const PagedArgs p, uint4* k, uint4* v,
                                                            int heads) {
  constexpr int LPR = D / 8;                       // lanes to a row
  constexpr int kPass = kMoveThreads / LPR;        // rows of one pass over the block
  constexpr int kPasses = kMoveTokens / kPass;     // passes to a head
  __shared__ TokenPlace place[kMoveTokens];
  __shared__ int coarse[kCoarse], lens[kCoarse];
  let_next_start();
  wait_for_previous();
  const int t0 = blockIdx.x * kMoveTokens;
  const int h0 = blockIdx.y * heads, h1 = min(h0 + heads, p.hkv);
  const int sub = threadIdx.x / LPR, l = threadIdx.x % LPR;
  // Rows of one head after another: everything steps by a constant. A thread's loads of kHeads heads
  // go out together, then they are converted and stored.
  constexpr int kHeads = 4 / kPasses;
  using Cell = typename std::conditional<kE4M3, uint2, uint4>::type;  // 8 channels in a page
  const long long page_step = 1ll << p.page_shift, row_step = static_cast<long long>(p.total_new) * LPR;
  uint4* mine[kPasses];
  uint4 x[kHeads][kPasses];
  uint32_t byte[kHeads][kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i)
    mine[i] = (blockIdx.z ? v : k) + (static_cast<long long>(h0) * p.total_new + t0 + i * kPass + sub) * LPR + l;
  auto load_rows = [&](int h) {
#pragma unroll
    for (int y = 0; y < kHeads; ++y)
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        x[y][i] = make_uint4(0u, 0u, 0u, 0u);
        if (t0 + i * kPass + sub < p.total_new && h + y < h1) x[y][i] = __ldcs(mine[i] + y * row_step);
      }
  };
  // Where a write's rows come from is known at once: the first are on their way while their places
  // are looked up.
  if constexpr (!kRead) load_rows(h0);
  find_places(p, t0, place, coarse, lens);
  if (blockIdx.x + blockIdx.y + blockIdx.z == 0)  // errors of sequences that no row is found in, too
    for (int i = threadIdx.x; i < p.n_seqs; i += kMoveThreads) seq_shape(p, i, true);
  bool at[kPasses];
  Cell* cells[kPasses];
  uint8_t* scales[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const TokenPlace r = place[i * kPass + sub];
    at[i] = r.page >= 0;
    const long long row = at[i] ? page_row(p, r.page, h0) + r.off : 0;
    cells[i] = reinterpret_cast<Cell*>(blockIdx.z ? p.v_pages : p.k_pages) + row * LPR + l;
    scales[i] = (blockIdx.z ? p.v_scales : p.k_scales) + row;
  }
  for (int h = h0; h < h1; h += kHeads) {
    if constexpr (!kRead) {
      if (h > h0) load_rows(h);
    } else {
#pragma unroll
      for (int y = 0; y < kHeads; ++y)
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
          x[y][i] = make_uint4(0u, 0u, 0u, 0u);
          byte[y][i] = 127u;
          if (!at[i] || h + y >= h1) continue;
          if constexpr (kE4M3) {
            const uint2 c = cells[i][y * page_step * LPR];
            x[y][i].x = c.x;
            x[y][i].y = c.y;
            byte[y][i] = scales[i][y * page_step];
          } else {
            x[y][i] = cells[i][y * page_step * LPR];
          }
        }
    }
#pragma unroll
    for (int y = 0; y < kHeads; ++y)
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const bool on = at[i] && h + y < h1;
        if constexpr (kRead) {
          if constexpr (kE4M3) x[y][i] = scaled8(make_uint2(x[y][i].x, x[y][i].y), e8m0_to_float(byte[y][i]));
          if (on) __stcs(mine[i] + y * row_step, x[y][i]);
        } else if constexpr (kE4M3) {
          const uint2 codes = quantise<LPR>(x[y][i], byte[y][i]);
          if (on) {
            cells[i][y * page_step * LPR] = codes;
            if (l == 0) scales[i][y * page_step] = static_cast<uint8_t>(byte[y][i]);
          }
        } else if (on) {
          cells[i][y * page_step * LPR] = x[y][i];
        }
      }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      mine[i] += kHeads * row_step;
      cells[i] += kHeads * page_step * LPR;
      scales[i] += kHeads * page_step;
    }
  }
}

// The launch overlaps the kernel before it in the stream where its blocks fill the GPU, so that this
// is worth the call's extra microsecond and a half on the host.
template <int D, bool kRead>
fcp_status launch_move(const PagedArgs& p, int dtype, void* k, void* v, cudaStream_t s) {
  const unsigned bx = static_cast<unsigned>((p.total_new + kMoveTokens - 1) / kMoveTokens);
  // all heads stay in one block while that leaves enough blocks for the GPU (4 sequences of up to
  // 16384 tokens written: 17.0 us; with a quarter of the heads to a block 32.2)
  int dev = 0, n_sm = 0;
  if (const fcp_status st = this_device(&dev, &n_sm); st != FCP_OK) return st;
  auto fills = [&](int heads) { return 2ll * bx * ((p.hkv + heads - 1) / heads) >= kEnough * n_sm; };
  int heads = p.hkv;
  while (heads > 1 && !fills(heads)) heads = (heads + 1) / 2;
  const dim3 grid(bx, static_cast<unsigned>((p.hkv + heads - 1) / heads), 2);
  uint4* pk = static_cast<uint4*>(k);
  uint4* pv = static_cast<uint4*>(v);
  auto* kernel = dtype == FCP_CACHE_E4M3 ? move_kernel<D, true, kRead> : move_kernel<D, false, kRead>;
  const char* where = kRead ? "cache read launch" : "cache write launch";
  if (fills(heads)) return launch_overlapped(kernel, grid, kMoveThreads, 0, s, where, p, pk, pv, heads);
  kernel<<<grid, kMoveThreads, 0, s>>>(p, pk, pv, heads);
  FCP_CUDA_TRY(cudaGetLastError(), where);
  return FCP_OK;
}

template <bool kRead>
fcp_status move(const fcp_cache* cache, const fcp_cache_batch* batch, void* k, void* v, void* stream) {
  PagedArgs p;
  if (const fcp_status st = paged_args(cache, batch, &p); st != FCP_OK) return st;
  if (p.total_new == 0 || p.n_seqs == 0) return FCP_OK;
  if (!k || !v || !aligned16(k) || !aligned16(v)) return FCP_ERR_INVALID;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cache->head_dim == 128 ? launch_move<128, kRead>(p, cache->dtype, k, v, s)
                                : launch_move<64, kRead>(p, cache->dtype, k, v, s);
}

}  // namespace
}  // namespace fcp

extern "C" fcp_status fcp_cache_write(const fcp_cache* cache, const fcp_cache_batch* batch, const void* k,
                                      const void* v, void* stream) {
  return fcp::move<false>(cache, batch, const_cast<void*>(k), const_cast<void*>(v), stream);
}

extern "C" fcp_status fcp_cache_read(const fcp_cache* cache, const fcp_cache_batch* batch, void* k, void* v,
                                     void* stream) {
  return fcp::move<true>(cache, batch, k, v, stream);
}
