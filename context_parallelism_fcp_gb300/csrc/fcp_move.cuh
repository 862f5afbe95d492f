// Shared by the kernels that move rows into and out of a paged cache: where a batch's packed rows lie,
// and the quantisation of a row.
#pragma once

#include "fcp_paged.h"

namespace fcp {

constexpr int kMoveThreads = 256;
constexpr int kMoveTokens = 32;   // packed rows of a block
constexpr int kCoarse = 1024;     // row offsets kept in shared memory

// The cache row (page * page_size + offset, to which a head adds its stride) of each of the
// block's tokens; -1 for rows behind the last sequence, rows before their sequence's first
// position and rows whose page is outside the cache. pos: the position; -1 for the first two of these.
struct TokenPlace {
  int32_t page, off, pos;
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
    const int pos = s.n > 0 ? s.len - s.n + (t - s.a) : -1;
    TokenPlace r{-1, 0, max(pos, -1)};
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

// The largest magnitudes of 8 bf16 channels as bf16 bits, of the even and of the odd ones: non-finite
// values order above every finite one.
__device__ __forceinline__ uint32_t top_pair(const uint4 x) {
  return max_u16x2(max_u16x2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), max_u16x2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
}

// Quantise 8 channels of a row whose largest magnitude is top: 8 codes and the row's scale byte.
__device__ __forceinline__ uint2 quantise8(const uint4 x, uint32_t top, uint32_t& scale_byte) {
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
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

// The same for the 8 channels of this lane, of a row shared by LPR lanes.
template <int LPR>
__device__ __forceinline__ uint2 quantise(const uint4 x, uint32_t& scale_byte) {
  uint32_t two = top_pair(x);
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) two = max_u16x2(two, __shfl_xor_sync(0xffffffffu, two, o));
  return quantise8(x, max(two & 0xffffu, two >> 16), scale_byte);
}

// Quantise 8 channels to e2m1, of 16 whose largest magnitude is top: 8 codes and the scale's byte.
// (Division by 6 and by the scale as products, rounded to 12 bits and to 2^-13: quotients that lie on a
// border between two codes become that border exactly, and others are at least 2^-9 of themselves away
// from one, since x has 8 significant bits and a border times a scale at most 7. So this rounds as the
// quotients themselves would.)
__device__ __forceinline__ uint32_t quantise4(const uint4 x, uint32_t top, float per_unit, uint32_t& scale_byte) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  const float sixth = __uint_as_float(top << 16) * per_unit * (1.f / 6.f);
  const float s = __uint_as_float((__float_as_uint(sixth) + 0x800u) & ~0xfffu);
  const uint32_t byte = max(static_cast<uint32_t>(__nv_cvt_float_to_fp8(s, __NV_SATFINITE, __NV_E4M3)), 1u);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(e4m3_to_float(byte)));
  inv *= per_unit;
  constexpr float kRound = 1536.f;  // 1.5 * 2^10: sums near it are multiples of 2^-13
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 y = dev::ffma2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u), inv, inv, kRound, kRound);
    y = dev::fadd2(y.x, y.y, -kRound, -kRound);
    asm("{\n.reg .b8 b;\n.reg .b16 h;\ncvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\nmov.b16 h, {b, 0};\ncvt.u32.u16 %0, h;\n}"
        : "=r"(c[i])
        : "f"(y.y), "f"(y.x));
  }
  const bool finite = top < 0x7f80u;
  scale_byte = finite ? byte : 0x7fu;
  return finite ? __byte_perm(__byte_perm(c[0], c[1], 0x3240), __byte_perm(c[2], c[3], 0x3240), 0x5410) : 0u;
}

}  // namespace fcp
