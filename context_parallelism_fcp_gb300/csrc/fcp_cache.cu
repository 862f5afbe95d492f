// Writing rows of K and V into the pages of a paged cache (quantising them where the cache is
// e4m3 or e2m1), and reading them back as bf16.
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
#include <cmath>
#include <type_traits>

#include "fcp_move.cuh"

namespace fcp {

static bool good_unit(float u) {
  int e = 0;
  return u > 0.f && std::isfinite(u) && std::frexp(u, &e) == 0.5f && e >= -59 && e <= 61;
}

fcp_status paged_args(const fcp_cache* c, const fcp_cache_batch* b, PagedArgs* out) {
  if (c == nullptr || b == nullptr || out == nullptr) return FCP_ERR_INVALID;
  if (c->n_pages < 0 || c->hkv <= 0 || c->page_size <= 0 || b->n_seqs < 0 || b->max_pages < 0 || b->total_new < 0 ||
      b->max_new < 0)
    return FCP_ERR_INVALID;
  if (c->dtype != FCP_CACHE_BF16 && c->dtype != FCP_CACHE_E4M3 && c->dtype != FCP_CACHE_E2M1) return FCP_ERR_INVALID;
  if (c->dtype == FCP_CACHE_E2M1 && !(good_unit(c->k_unit) && good_unit(c->v_unit))) return FCP_ERR_INVALID;
  if (c->head_dim != 64 && c->head_dim != 128) return FCP_ERR_UNSUPPORTED;
  if (c->page_size < 16 || c->page_size > 4096 || (c->page_size & (c->page_size - 1)) != 0) return FCP_ERR_UNSUPPORTED;
  if (static_cast<long long>(b->max_pages) * c->page_size > 1ll << 30) return FCP_ERR_UNSUPPORTED;
  if (b->n_seqs > 65536 || b->total_new > 1 << 30) return FCP_ERR_UNSUPPORTED;
  if (c->status == nullptr || !aligned16(c->status)) return FCP_ERR_INVALID;
  if (b->n_seqs > 0 && (!b->cu_new || !b->lens || (b->max_pages > 0 && !b->block_table))) return FCP_ERR_INVALID;
  if (!aligned4(b->cu_new) || !aligned4(b->lens) || !aligned4(b->block_table)) return FCP_ERR_INVALID;
  if (c->n_pages > 0) {
    if (!c->k_pages || !c->v_pages || !aligned16(c->k_pages) || !aligned16(c->v_pages)) return FCP_ERR_INVALID;
    if (c->dtype != FCP_CACHE_BF16 &&
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
  p.k_unit = c->dtype == FCP_CACHE_E2M1 ? c->k_unit : 1.f;
  p.v_unit = c->dtype == FCP_CACHE_E2M1 ? c->v_unit : 1.f;
  if (c->n_pages == 0) p.k_pages = p.v_pages = p.k_scales = p.v_scales = reinterpret_cast<uint8_t*>(c->status);
  *out = p;
  return FCP_OK;
}

namespace {

constexpr int kEnough = 8;        // blocks of an SM: all that its threads allow

// grid (ceil(T / 32), ceil(Hkv / heads per block), 2: K or V)
template <int D, int kKind, bool kRead>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const PagedArgs p, uint4* k, uint4* v,
                                                            int heads) {
  constexpr bool kE4M3 = kKind == FCP_CACHE_E4M3, kE2M1 = kKind == FCP_CACHE_E2M1;
  constexpr int kScales = kE2M1 ? D / 16 : 1;      // scales of a row
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
  using Cell = std::conditional_t<kE2M1, uint32_t, std::conditional_t<kE4M3, uint2, uint4>>;  // 8 channels in a page
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
    scales[i] = (blockIdx.z ? p.v_scales : p.k_scales) + row * kScales + (kE2M1 ? l / 2 : 0);
  }
  [[maybe_unused]] const float unit = blockIdx.z ? p.v_unit : p.k_unit;
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
          } else if constexpr (kE2M1) {
            x[y][i].x = cells[i][y * page_step * LPR];
            byte[y][i] = scales[i][y * page_step * kScales];
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
          if constexpr (kE2M1) x[y][i] = scaled8(x[y][i].x, e4m3_to_float(byte[y][i]) * unit);
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
      scales[i] += kHeads * page_step * kScales;
    }
  }
}

// Writing e2m1 rows: as above with 16 channels, one scale's, to a thread. Bound by the instructions of the
// quantisation about as much as by HBM: 14000 tokens of 8 heads take 15.2 us (4870 GB/s), with 8 channels to
// a thread 18.4; reading them back, 8 channels to a thread, takes 14.8.
template <int D>
__global__ void __launch_bounds__(kMoveThreads) store4_kernel(const PagedArgs p, const uint4* k, const uint4* v,
                                                              int heads) {
  constexpr int kLanes = D / 16, kGroups = kMoveThreads / (kLanes * kMoveTokens);  // threads of a row; heads at a time
  constexpr int kHeads = 4;  // rows that a thread has in flight
  __shared__ TokenPlace place[kMoveTokens];
  __shared__ int coarse[kCoarse], lens[kCoarse];
  let_next_start();
  wait_for_previous();
  const int t0 = blockIdx.x * kMoveTokens;
  const int l = threadIdx.x % kLanes, tok = threadIdx.x / kLanes % kMoveTokens, group = threadIdx.x / (kLanes * kMoveTokens);
  const int h0 = blockIdx.y * heads + group, h1 = min(static_cast<int>(blockIdx.y + 1) * heads, p.hkv);
  const long long row_step = static_cast<long long>(p.total_new) * (2 * kLanes);
  const uint4* src = (blockIdx.z ? v : k) + static_cast<long long>(t0 + tok) * (2 * kLanes) + 2 * l;
  uint4 x[kHeads][2];
  auto load_rows = [&](int h) {
#pragma unroll
    for (int y = 0; y < kHeads; ++y) {
      x[y][0] = x[y][1] = make_uint4(0u, 0u, 0u, 0u);
      if (t0 + tok < p.total_new && h + y * kGroups < h1) {
        x[y][0] = __ldcs(src + (h + y * kGroups) * row_step);
        x[y][1] = __ldcs(src + (h + y * kGroups) * row_step + 1);
      }
    }
  };
  load_rows(h0);
  find_places(p, t0, place, coarse, lens);
  if (blockIdx.x + blockIdx.y + blockIdx.z == 0)  // errors of sequences that no row is found in, too
    for (int i = threadIdx.x; i < p.n_seqs; i += kMoveThreads) seq_shape(p, i, true);
  const TokenPlace at = place[tok];
  const float per_unit = 1.f / (blockIdx.z ? p.v_unit : p.k_unit);  // exact: powers of two
  uint2* cells = reinterpret_cast<uint2*>(blockIdx.z ? p.v_pages : p.k_pages);
  uint8_t* scales = blockIdx.z ? p.v_scales : p.k_scales;
  for (int h = h0; h < h1; h += kHeads * kGroups) {
    if (h > h0) load_rows(h);
#pragma unroll
    for (int y = 0; y < kHeads; ++y) {
      const uint32_t two = max_u16x2(top_pair(x[y][0]), top_pair(x[y][1])), top = max(two & 0xffffu, two >> 16);
      uint32_t byte;
      const uint32_t lo = quantise4(x[y][0], top, per_unit, byte), hi = quantise4(x[y][1], top, per_unit, byte);
      if (at.page >= 0 && h + y * kGroups < h1) {
        const long long cell = (page_row(p, at.page, h + y * kGroups) + at.off) * kLanes + l;
        cells[cell] = make_uint2(lo, hi);
        scales[cell] = static_cast<uint8_t>(byte);
      }
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
  if constexpr (!kRead) {
    if (dtype == FCP_CACHE_E2M1) {
      const uint4 *ck = pk, *cv = pv;
      if (fills(heads)) return launch_overlapped(store4_kernel<D>, grid, kMoveThreads, 0, s, "cache write launch", p, ck, cv, heads);
      store4_kernel<D><<<grid, kMoveThreads, 0, s>>>(p, ck, cv, heads);
      FCP_CUDA_TRY(cudaGetLastError(), "cache write launch");
      return FCP_OK;
    }
  }
  auto* kernel = dtype == FCP_CACHE_E4M3 ? move_kernel<D, FCP_CACHE_E4M3, kRead> : move_kernel<D, FCP_CACHE_BF16, kRead>;
  if constexpr (kRead) {
    if (dtype == FCP_CACHE_E2M1) kernel = move_kernel<D, FCP_CACHE_E2M1, true>;
  }
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
