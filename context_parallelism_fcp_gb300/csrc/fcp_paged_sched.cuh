// How the attention over a paged cache is split over the GPU, and the merge of what is split.
//
// The work is a list of groups in the order sequence, KV head, unit: a unit is the largest set
// of (new token, query head) rows that one block handles together, and a group reads the keys
// [0, end) that any row of its unit sees, in granules of 128. Laid end to end, the groups'
// granules form one line, and block b of B takes the b-th of B equal shares of it. So the load
// is even whatever the lengths are, no block ever holds more than two groups that it does not
// finish (its first and its last), and the space for partial results does not depend on the
// batch. Every block derives its share from the lengths in device memory, so a captured graph
// follows them.
#pragma once

#include "fcp_paged.h"
#include "fcp_sm100.cuh"

namespace fcp {

constexpr int kGranule = 128;  // keys

struct AttnArgs {
  PagedArgs c;
  int32_t group;       // query heads of one KV head
  int32_t causal;
  float scale_log2;
  __nv_bfloat16* o;    // [Hq, T, D]
  float* lse;          // [Hq, T]
  float* part_o;       // [2 * blocks, kRows, D] unnormalised sums
  float2* part_ml;     // [2 * blocks, kRows] (row maximum in log2 units, row sum)
  const __nv_bfloat16* q;
};

// First key that no row of a unit ending with new token `last` sees.
__device__ __forceinline__ int key_end(const SeqShape& s, int last, int causal) {
  return causal ? max(0, s.len - s.n + min(last, s.n - 1) + 1) : s.len;
}
__device__ __forceinline__ int granules_of(int end) { return max(1, (end + kGranule - 1) / kGranule); }

// Units of a policy: units(s, group) and granules(s, group, unit, causal).
//
// Few rows: row r of a KV head is (new token r / group, head r % group); a unit is kRows of them.
template <int kRowsPerUnit>
struct FewRows {
  static constexpr int kRows = kRowsPerUnit;
  static __device__ __forceinline__ int units(const SeqShape& s, int group) {
    return static_cast<int>((static_cast<long long>(s.n) * group + kRows - 1) / kRows);
  }
  static __device__ __forceinline__ int end(const SeqShape& s, int group, int u, int causal) {
    return key_end(s, static_cast<int>(((u + 1ll) * kRows - 1) / group), causal);
  }
  // (token, head of the group) of row r of unit u; false behind the last
  static __device__ __forceinline__ bool row(const SeqShape& s, int group, int u, int r, int& tok, int& head) {
    const long long x = static_cast<long long>(u) * kRows + r;
    tok = static_cast<int>(x / group);
    head = static_cast<int>(x - static_cast<long long>(tok) * group);
    return tok < s.n;
  }
};

// The group at a block's current place on the line.
template <class P>
struct Walk {
  int i, h, u, n_units, end, g;   // sequence, KV head, unit, units a head, keys, granules
  SeqShape s;
  long long f0;                   // the group's first granule on the line

  __device__ __forceinline__ void enter(const AttnArgs& a) {
    end = P::end(s, a.group, u, a.causal);
    g = granules_of(end);
  }
  __device__ __forceinline__ void next(const AttnArgs& a) {
    f0 += g;
    if (++u == n_units) {
      u = 0;
      if (++h == a.c.hkv) {
        h = 0;
        do {
          if (++i >= a.c.n_seqs) return;
          s = seq_shape(a.c, i, false);
        } while (s.n == 0);
        n_units = P::units(s, a.group);
      }
    }
    enter(a);
  }
};

template <class P>
__device__ __forceinline__ long long head_granules(const AttnArgs& a, const SeqShape& s) {
  long long sum = 0;
  const int n = P::units(s, a.group);
  for (int u = 0; u < n; ++u) sum += granules_of(P::end(s, a.group, u, a.causal));
  return sum;
}

// Shared memory of the line's prefix sums: thread t's sequences begin at prefix[t].
template <int kThreads>
struct Line {
  long long prefix[kThreads + 1];
  long long warp_sum[kThreads / 32];
  int per;  // sequences to a thread
};

// All kThreads threads; ends with a barrier.
template <class P, int kThreads>
__device__ __forceinline__ void build_line(const AttnArgs& a, Line<kThreads>& line, bool report) {
  const int per = (a.c.n_seqs + kThreads - 1) / kThreads;
  long long mine = 0;
  for (int i = threadIdx.x * per; i < min((static_cast<int>(threadIdx.x) + 1) * per, a.c.n_seqs); ++i) {
    const SeqShape s = seq_shape(a.c, i, report);
    if (s.n > 0) mine += head_granules<P>(a, s) * a.c.hkv;
  }
  long long x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if ((threadIdx.x & 31) >= o) x += y;
  }
  if ((threadIdx.x & 31) == 31) line.warp_sum[threadIdx.x >> 5] = x;
  __syncthreads();
  for (int w = 0; w < static_cast<int>(threadIdx.x >> 5); ++w) x += line.warp_sum[w];
  line.prefix[threadIdx.x + 1] = x;
  if (threadIdx.x == 0) {
    line.prefix[0] = 0;
    line.per = per;
  }
  __syncthreads();
}

// Place `w` on the group that holds granule f of the line (f < the line's length). False only
// if the lengths no longer are what the line was built from.
template <class P, int kThreads>
__device__ __forceinline__ bool seek(const AttnArgs& a, const Line<kThreads>& line, long long f, Walk<P>& w) {
  int lo = 0, hi = kThreads;  // prefix[lo] <= f < prefix[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (line.prefix[mid] <= f) lo = mid; else hi = mid;
  }
  w.i = lo * line.per;
  w.f0 = line.prefix[lo];
  long long per_head;
  while (true) {
    if (w.i >= a.c.n_seqs) return false;
    w.s = seq_shape(a.c, w.i, false);
    per_head = w.s.n > 0 ? head_granules<P>(a, w.s) : 0;
    if (f < w.f0 + per_head * a.c.hkv) break;
    w.f0 += per_head * a.c.hkv;
    ++w.i;
  }
  w.h = static_cast<int>((f - w.f0) / per_head);
  w.f0 += w.h * per_head;
  w.n_units = P::units(w.s, a.group);
  w.u = 0;
  w.enter(a);
  while (f >= w.f0 + w.g) {
    w.f0 += w.g;
    ++w.u;
    w.enter(a);
  }
  return true;
}

__device__ __forceinline__ long long share_begin(long long total, int b, int blocks) {
  return total / blocks * b + total % blocks * b / blocks;
}

// Where a block's piece [ga, gb) of a group of g granules goes: the output itself when it is the
// whole group, else the block's slot for a group it continues (0) or begins (1).
__device__ __forceinline__ int piece_slot(int b, int ga, int gb, int g) {
  return ga == 0 && gb == g ? -1 : 2 * b + (ga == 0 ? 1 : 0);
}

// Joins the pieces of the group that block b of the attention begins and does not finish: with
// M the largest of the pieces' maxima, O = sum 2^(m - M) o / sum 2^(m - M) l. grid (blocks,
// row slices): the pieces are read once, from L2, and most blocks find nothing to join.
template <class P, int D>
__global__ void __launch_bounds__(128) paged_merge_kernel(const AttnArgs a, int blocks) {
  __shared__ Line<128> line;
  const int b = blockIdx.x;
  build_line<P, 128>(a, line, false);
  const long long total = line.prefix[128];
  const long long w0 = share_begin(total, b, blocks), w1 = share_begin(total, b + 1, blocks);
  Walk<P> w;
  const bool mine = w0 < w1 && w1 < total && seek<P, 128>(a, line, w1 - 1, w) && w.f0 >= w0 && w.f0 + w.g > w1;
  // the pieces are written (every block waits, so that this grid never ends before the attention)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!mine) return;
  int last = b + 1;
  while (last + 1 < blocks && share_begin(total, last + 1, blocks) < w.f0 + w.g) ++last;

  constexpr int kLanes = D / 4;              // threads to a row, 4 channels each
  constexpr int kPer = 128 / kLanes;         // rows at a time
  const int lane = threadIdx.x % kLanes;
  for (int r = blockIdx.y * kPer + threadIdx.x / kLanes; r < P::kRows; r += kPer * gridDim.y) {
    int tok, head;
    if (!P::row(w.s, a.group, w.u, r, tok, head)) continue;
    float m = -INFINITY;
    for (int x = b; x <= last; ++x) {
      if (x > b && share_begin(total, x, blocks) == share_begin(total, x + 1, blocks)) continue;
      m = fmaxf(m, __ldcg(&a.part_ml[static_cast<long long>(2 * x + (x == b)) * P::kRows + r].x));
    }
    const float mb = m == -INFINITY ? 0.f : m;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    for (int x = b; x <= last; ++x) {
      if (x > b && share_begin(total, x, blocks) == share_begin(total, x + 1, blocks)) continue;
      const long long at = static_cast<long long>(2 * x + (x == b)) * P::kRows + r;
      const float2 ml = __ldcg(&a.part_ml[at]);
      const float f = exp2f(ml.x - mb);
      const float4 y = __ldcg(reinterpret_cast<const float4*>(a.part_o + at * D) + lane);
      l = fmaf(f, ml.y, l);
      acc.x = fmaf(f, y.x, acc.x);
      acc.y = fmaf(f, y.y, acc.y);
      acc.z = fmaf(f, y.z, acc.z);
      acc.w = fmaf(f, y.w, acc.w);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const long long row = static_cast<long long>(w.h * a.group + head) * a.c.total_new + w.s.a + tok;
    uint2 pk;
    pk.x = dev::pack_bf16(acc.x * inv, acc.y * inv);
    pk.y = dev::pack_bf16(acc.z * inv, acc.w * inv);
    reinterpret_cast<uint2*>(a.o + row * D)[lane] = pk;
    if (lane == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
  }
}

}  // namespace fcp
