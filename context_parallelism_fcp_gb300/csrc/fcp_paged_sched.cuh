// How the attention over a paged cache is split over the GPU, and the merge of what is split.
//
// The work is a list of groups in the order sequence, KV head, unit: a unit is the largest set
// of (new token, query head) rows that one block handles together, and a group reads the keys
// [0, end) that any row of its unit sees, in granules of 128. Laid end to end, the groups form
// one line, each as long as its granules and the policy's kOverhead in front of them (what
// loading its rows and storing their results costs, in granules), and block b of B takes the
// b-th of B equal shares of it. So the load is even whatever the lengths are, no block ever
// holds more than two groups that it does not finish (its first and its last), and the space
// for partial results does not depend on the batch. Every block derives its share from the
// lengths in device memory, so a captured graph follows them.
#pragma once

#include "fcp_paged.h"
#include "fcp_sm100.cuh"

namespace fcp {

constexpr int kGranule = 128;    // keys
constexpr int kMaxBlocks = 640;       // few rows: up to four blocks to each of up to 160 SMs
constexpr int kMaxChunkBlocks = 160;  // chunks: one

struct SplitGroup;

struct AttnArgs {
  PagedArgs c;
  int32_t group;       // query heads of one KV head
  int32_t causal;
  float scale_log2;
  __nv_bfloat16* o;    // [Hq, T, D]
  float* lse;          // [Hq, T]
  float* part_o;       // [2 * blocks, kRows, D] unnormalised sums
  float2* part_ml;     // [2 * blocks, kRows] (row maximum in log2 units, row sum)
  SplitGroup* split;     // [blocks]
  const __nv_bfloat16* q;
  // Little work at most: the call after this one may start while the merge runs. (4 sequences of up
  // to 333 keys, call after call: 8.6 us instead of 10.4; with 128 of up to 8192 the next call's
  // early blocks were in the way: 180 us instead of 171.) The host knows no lengths, only how many
  // positions the block table has room for.
  int32_t small;
};

// a / b of lengths that nearly always fit 32 bits.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// First key that no row of a unit ending with new token `last` sees.
__device__ __forceinline__ int key_end(const SeqShape& s, int last, int causal) {
  return causal ? max(0, s.len - s.n + min(last, s.n - 1) + 1) : s.len;
}
__device__ __forceinline__ int granules_of(int end) { return max(1, (end + kGranule - 1) / kGranule); }

// Units of a policy: units(s, group) and granules(s, group, unit, causal).
//
// Few rows: row r of a KV head is (new token r / group, head r % group); a unit is kRows of them.
template <int kRowsPerUnit, int kOverheadGranules = 1>
struct FewRows {
  static constexpr int kRows = kRowsPerUnit;
  // A block's share is two granules at least: finer pieces cost more in the merge than they save (40
  // sequences of up to 3000 keys of one KV head 27.8 us with 1, 15.5 with 2, 16.7 with 3; 10 of up to
  // 1000, 4 KV heads: 13.7, 11.0, 11.5).
  static constexpr int kLeastShare = 2;
  static constexpr int kWarpPieces = 8;  // of a row, up to which the merge gives a row to a warp
  static constexpr int kOverhead = kOverheadGranules;
  static __device__ __forceinline__ int units(const SeqShape& s, int group) {
    return static_cast<int>((static_cast<long long>(s.n) * group + kRows - 1) / kRows);
  }
  // All of the sequence's keys: the mask leaves the last few out where that matters.
  static __device__ __forceinline__ int end(const SeqShape& s, int, int, int) { return s.len; }
  static __device__ __forceinline__ long long head_length(const SeqShape& s, int group, int) {
    return static_cast<long long>(units(s, group)) * (kOverhead + granules_of(s.len));
  }
  // The unit of a head that holds place f >= f0 of the line, where the head begins at f0; f0
  // becomes where the unit begins.
  static __device__ __forceinline__ int find(const SeqShape& s, int, int, long long f, long long& f0) {
    const int len = kOverhead + granules_of(s.len);
    if (f < f0 + len) return 0;
    const int u = static_cast<int>(quotient(f - f0, len));
    f0 += static_cast<long long>(u) * len;
    return u;
  }
  // (token, head of the group) of row r of unit u; false behind the last
  static __device__ __forceinline__ bool row(const SeqShape& s, int group, int u, int r, int& tok, int& head) {
    const long long x = static_cast<long long>(u) * kRows + r;
    tok = static_cast<int>(quotient(x, group));
    head = static_cast<int>(x - static_cast<long long>(tok) * group);
    return tok < s.n;
  }
};

// Chunks: a tile is 128 rows of a KV head, 2^log_tokens new tokens of each of 128 / 2^log_tokens query
// heads, head by head. Whole 128s of tokens make tiles of one head each, the tokens that are left
// tiles of 128, 64, 32 or 16 tokens, so that short chunks and remainders fill tiles with heads
// instead of padding. Tiles are ordered tokens first, heads within them, and a unit is two (kTiles), or
// one for batches whose sequences have no more rows than that.
template <int kTilesPerUnit>
struct ChunkRowsOf {
  static constexpr int kTiles = kTilesPerUnit;
  static constexpr int kRows = kTiles * kTileM;
  static constexpr int kLeastShare = 1;  // 4, 6 and 8 were slower on every small batch tried
  static constexpr int kWarpPieces = 32;
  // One value for all caches and both sizes of unit. (With 3, 5, 8, 4 bits, units of one tile as the others then: 9 mixed
  // chunks 51.7, 50.6, 49.2 us; 16 chunks of 512 with nothing before them 221, 224, 223; 16 x 5 tokens over up to
  // 8192 keys 335, 346, 362. Larger values for units of two tiles alone were not measured.)
  static constexpr int kOverhead = 3;
  struct Tile {
    int tok0, log_tokens, head0;
    // (token, head of the group) of row r; false for rows of no token or head
    __device__ __forceinline__ bool row(const SeqShape& s, int group, int r, int& tok, int& head) const {
      tok = tok0 + (r & ((1 << log_tokens) - 1));
      head = head0 + (r >> log_tokens);
      return tok < s.n && head < group;
    }
  };
  struct Shape {
    int n128, full, log_rest, tiles;  // whole 128s of tokens, their tiles; the rest's tokens; all tiles
    __device__ __forceinline__ Shape(const SeqShape& s, int group) {
      const int rest = s.n & 127;
      n128 = s.n >> 7;
      full = n128 * group;
      log_rest = rest > 64 ? 7 : (rest > 32 ? 6 : (rest > 16 ? 5 : 4));
      tiles = full + (rest > 0 ? (group + (kTileM >> log_rest) - 1) >> (7 - log_rest) : 0);
    }
    __device__ __forceinline__ Tile tile(int x, int group) const {
      if (x >= full) return Tile{n128 << 7, log_rest, (x - full) << (7 - log_rest)};
      const int tt = x / group;
      return Tile{tt << 7, 7, x - tt * group};
    }
    // Units whose last tile comes before token tile tt (n128: the rest).
    __device__ __forceinline__ int first_unit(int tt, int group) const {
      return tt > n128 ? (tiles + kTiles - 1) / kTiles : tt * group / kTiles;
    }
  };
  // Length on the line of a unit whose last tile is of token tile tt.
  static __device__ __forceinline__ int length(const SeqShape& s, int tt, int causal) {
    return kOverhead + granules_of(key_end(s, (tt << 7) + 127, causal));
  }
  static __device__ __forceinline__ int units(const SeqShape& s, int group) { return (Shape(s, group).tiles + kTiles - 1) / kTiles; }
  static __device__ __forceinline__ int tiles_of(const SeqShape& s, int group, int u) {
    return min(kTiles, Shape(s, group).tiles - kTiles * u);
  }
  static __device__ __forceinline__ int end(const SeqShape& s, int group, int u, int causal) {
    const Shape z(s, group);
    const int x = min(kTiles * u + kTiles - 1, z.tiles - 1);
    return key_end(s, ((x < z.full ? x / group : z.n128) << 7) + 127, causal);
  }
  static __device__ __forceinline__ long long head_length(const SeqShape& s, int group, int causal) {
    const Shape z(s, group);
    long long sum = 0;
    for (int tt = 0, u = 0; tt <= z.n128; ++tt) {
      const int next = z.first_unit(tt + 1, group);
      sum += static_cast<long long>(next - u) * length(s, tt, causal);
      u = next;
    }
    return sum;
  }
  static __device__ __forceinline__ int find(const SeqShape& s, int group, int causal, long long f, long long& f0) {
    const Shape z(s, group);
    for (int tt = 0, u = 0;; ++tt) {
      const int next = z.first_unit(tt + 1, group), len = length(s, tt, causal);
      const long long behind = f0 + static_cast<long long>(next - u) * len;
      if (f < behind) {
        const int x = static_cast<int>(quotient(f - f0, len));
        f0 += static_cast<long long>(x) * len;
        return u + x;
      }
      f0 = behind;
      u = next;
    }
  }
  static __device__ __forceinline__ bool row(const SeqShape& s, int group, int u, int r, int& tok, int& head) {
    const Shape z(s, group);
    const int x = kTiles * u + (r >> 7);
    return x < z.tiles && z.tile(x, group).row(s, group, r & (kTileM - 1), tok, head);
  }
};
using ChunkRows = ChunkRowsOf<2>;

// What each warp's sequences add to the line, and how many those are.
template <int kThreads>
struct Line {
  static constexpr int kWarps = kThreads / 32;
  long long warp_sum[kWarps];
  __device__ __forceinline__ static int per_thread(int n_seqs) { return (n_seqs + kThreads - 1) / kThreads; }
};

// The group at a block's current place on the line.
template <class P>
struct Walk {
  int i, h, u, n_units, end, g;   // sequence, KV head, unit, units a head, keys, granules
  SeqShape s;
  long long f0;                   // where the group begins on the line

  __device__ __forceinline__ void enter(const AttnArgs& a) {
    end = P::end(s, a.group, u, a.causal);
    g = granules_of(end);
  }
  __device__ __forceinline__ long long behind() const { return f0 + P::kOverhead + g; }
  // Granules [ga, gb) of the group that the part [w0, w1) of the line holds.
  __device__ __forceinline__ void part(long long w0, long long w1, int& ga, int& gb) const {
    ga = static_cast<int>(max(w0 - f0 - P::kOverhead, 0ll));
    gb = static_cast<int>(min(max(w1 - f0 - P::kOverhead, 0ll), static_cast<long long>(g)));
  }
  // To the next group, or just behind this one where that is the share's end w1.
  template <int kThreads>
  __device__ __forceinline__ void next(const AttnArgs& a, const Line<kThreads>& line, long long w1) {
    f0 = behind();
    if (f0 >= w1) return;
    if (++u == n_units) {
      u = 0;
      if (++h == a.c.hkv) {
        h = 0;
        if (++i < a.c.n_seqs) s = seq_shape(a.c, i, false);
        if (i < a.c.n_seqs && s.n == 0) skip(a, line);
        if (i >= a.c.n_seqs) return;
        n_units = P::units(s, a.group);
      }
    }
    enter(a);
  }
  // From a sequence without a new token to the next with one, whose groups begin at f0: past the warps
  // whose sequences end before that, then 8 offsets at a time. (One sequence at a time, and on past the
  // share's end, 30000 idle sequences between busy ones took 3.1 ms; now 0.17 ms for single tokens.)
  template <int kThreads>
  __device__ __forceinline__ void skip(const AttnArgs& a, const Line<kThreads>& line) {
    int w = 0;
    for (long long at = line.warp_sum[0]; at <= f0 && w + 1 < Line<kThreads>::kWarps; at += line.warp_sum[w]) ++w;
    i = max(i + 1, w * 32 * Line<kThreads>::per_thread(a.c.n_seqs));
    while (i < a.c.n_seqs) {
      constexpr int kAhead = 8;
      int cu[kAhead + 1], x = kAhead;
#pragma unroll
      for (int y = 0; y <= kAhead; ++y) cu[y] = load(a.c.cu + min(i + y, a.c.n_seqs));
#pragma unroll
      for (int y = kAhead - 1; y >= 0; --y) x = cu[y] < cu[y + 1] ? y : x;
      i += x;
      if (x == kAhead) continue;
      s = seq_shape(a.c, i, false);
      if (s.n > 0) return;
      ++i;
    }
  }
};

// The blocks' shares of a line of length `total`: block b < blocks takes [begin(b), begin(b + 1)),
// which is not empty (blocks is less than the grid where the line is shorter).
struct Shares {
  long long total;
  int blocks;
  __device__ __forceinline__ Shares(long long line, int grid, int least)
      : total(line), blocks(static_cast<int>(min((line + least - 1) / least, static_cast<long long>(grid)))) {}
  __device__ __forceinline__ long long begin(int b) const { return quotient(total * b, blocks); }
  // The block that takes place f: the last b with total * b / blocks < f + 1.
  __device__ __forceinline__ int owner(long long f) const {
    return static_cast<int>(quotient((f + 1) * blocks - 1, total));
  }
};

// Builds the line, and calls place(walk, shares, w0, w1) with the walk on the group that holds the
// beginning w0 of this block's share [w0, w1): each thread adds up its sequences, and the thread that
// finds the place among its own makes the call, with the lengths it already has. A block without a
// share (blocks <= its index) makes none. All kThreads threads; ends with a barrier. report: record
// the batch's errors. (The chain from the lengths to the first keys is most of a small call's
// time: that the finder also works out the first piece, with few divisions in a row, took
// 10 sequences of up to 1000 tokens from 9.1 to 8.6 us.)
template <class P, int kThreads, class Place>
__device__ __forceinline__ Shares begin_walk(const AttnArgs& a, Line<kThreads>& line, bool report, Place place) {
  const int tid = threadIdx.x, per = Line<kThreads>::per_thread(a.c.n_seqs);
  const int i0 = tid * per, i1 = min(i0 + per, a.c.n_seqs);
  SeqShape s{0, 0, 0};
  long long mine = 0, per_head = 0;
  for (int i = i0; i < i1; ++i) {
    s = seq_shape(a.c, i, report);
    per_head = s.n > 0 ? P::head_length(s, a.group, a.causal) : 0;
    mine += per_head * a.c.hkv;
  }
  long long behind = mine;  // where this thread's sequences end on the line
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, behind, o);
    if ((tid & 31) >= o) behind += y;
  }
  if ((tid & 31) == 31) line.warp_sum[tid >> 5] = behind;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w == (tid >> 5)) behind += total;
    total += line.warp_sum[w];
  }
  const Shares sh(total, gridDim.x, P::kLeastShare);
  const int b = blockIdx.x;
  if (b < sh.blocks) {
    const long long f = sh.begin(b), f1 = sh.begin(b + 1);
    if (behind - mine <= f && f < behind) {
      Walk<P> w;
      w.f0 = behind - mine;
      for (w.i = i0; w.i < i1; ++w.i) {
        w.s = s;
        if (per > 1) {
          w.s = seq_shape(a.c, w.i, false);
          if (w.s.n == 0) continue;
          per_head = P::head_length(w.s, a.group, a.causal);
        }
        if (f >= w.f0 + per_head * a.c.hkv) {
          w.f0 += per_head * a.c.hkv;
          continue;
        }
        w.h = static_cast<int>(quotient(f - w.f0, per_head));
        w.f0 += w.h * per_head;
        w.n_units = P::units(w.s, a.group);
        w.u = P::find(w.s, a.group, a.causal, f, w.f0);
        w.enter(a);
        place(w, sh, f, f1);
        break;
      }
    }
  }
  __syncthreads();
  return sh;
}

// Where a block's piece [ga, gb) of a group of g granules goes: the output itself when it is the
// whole group, else the block's slot for a group it continues (0) or begins (1).
__device__ __forceinline__ int piece_slot(int b, int ga, int gb, int g) {
  return ga == 0 && gb == g ? -1 : 2 * b + (ga == 0 ? 1 : 0);
}

// The group that a block begins and does not finish, for the merge: blocks (b, last] continue it
// (last = b: there is none).
struct SplitGroup {
  int32_t last, a, n, h, u;
  int32_t reserved[3];
};
static_assert(sizeof(SplitGroup) == 32, "two 16-byte loads");

// Joins the pieces of the groups that blocks split: with M the largest of a row's maxima,
// O = sum 2^(m - M) o / sum 2^(m - M) l, over the pieces in a fixed order. grid (blocks, row
// slices); a warp takes rows of up to kWarpPieces pieces, the whole block a row of more. Bound by
// latency: what is read is 2 * blocks partial results at most, 5 MB for single tokens (9 us on its
// own and cold, of which a call that follows its attention in the stream sees 3 to 4).
constexpr int kMergeWarps = 4;
template <class P, int D>
__global__ void __launch_bounds__(32 * kMergeWarps) paged_merge_kernel(const AttnArgs a) {
  constexpr int kPieceLanes = D / 4;                             // lanes of a piece, 4 channels each
  constexpr int kAtOnce = kMergeWarps * 32 / kPieceLanes;        // pieces at a time
  __shared__ float weight[kMaxBlocks];
  __shared__ float2 warp_ml[kMergeWarps];
  __shared__ float4 part[kAtOnce][kPieceLanes];
  const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  wait_for_previous();
  if (a.small) let_next_start();
  const SplitGroup g = a.split[b];
  const int count = g.last - b + 1;
  if (count <= 1) return;
  const SeqShape s{g.a, g.n, 0};
  if (count <= P::kWarpPieces) {
    // a warp takes two rows on its own, the loads of four pieces of both side by side
    constexpr int kEach = D / 32;  // channels of a lane
    constexpr int kR = 2, kX = 4;
    const int stride = gridDim.y * kMergeWarps;
    for (int r0 = blockIdx.y * kMergeWarps + warp; r0 < P::kRows; r0 += kR * stride) {
      float m[kR], l[kR], acc[kR][kEach];
      long long out[kR];  // output row; -1: none
#pragma unroll
      for (int k = 0; k < kR; ++k) {
        int tok, head;
        const int r = r0 + k * stride;
        const bool on = r < P::kRows && P::row(s, a.group, g.u, r, tok, head);
        out[k] = on ? static_cast<long long>(g.h * a.group + head) * a.c.total_new + s.a + tok : -1;
        m[k] = -INFINITY;
        l[k] = 0.f;
#pragma unroll
        for (int e = 0; e < kEach; ++e) acc[k][e] = 0.f;
      }
      for (int x0 = 0; x0 < count; x0 += kX) {
        float2 ml[kX][kR];
        float y[kX][kR][kEach];
#pragma unroll
        for (int q = 0; q < kX; ++q)
#pragma unroll
          for (int k = 0; k < kR; ++k) {
            ml[q][k] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int e = 0; e < kEach; ++e) y[q][k][e] = 0.f;
            if (x0 + q < count && out[k] >= 0) {
              const long long at = static_cast<long long>(2 * (b + x0 + q) + (x0 + q == 0)) * P::kRows + r0 + k * stride;
              ml[q][k] = a.part_ml[at];
#pragma unroll
              for (int e = 0; e < kEach; e += 2)
                *reinterpret_cast<float2*>(&y[q][k][e]) = *reinterpret_cast<const float2*>(a.part_o + at * D + lane * kEach + e);
            }
          }
#pragma unroll
        for (int k = 0; k < kR; ++k) {
          float top = m[k];
#pragma unroll
          for (int q = 0; q < kX; ++q) top = fmaxf(top, ml[q][k].x);
          const float mb = top == -INFINITY ? 0.f : top;
          const float f0 = exp2f(m[k] - mb);
          m[k] = top;
          l[k] *= f0;
#pragma unroll
          for (int e = 0; e < kEach; ++e) acc[k][e] *= f0;
#pragma unroll
          for (int q = 0; q < kX; ++q) {
            const float f = exp2f(ml[q][k].x - mb);
            l[k] = fmaf(f, ml[q][k].y, l[k]);
#pragma unroll
            for (int e = 0; e < kEach; ++e) acc[k][e] = fmaf(f, y[q][k][e], acc[k][e]);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kR; ++k)
        if (out[k] >= 0) {
          const float inv = l[k] == 0.f ? 0.f : 1.f / l[k];
#pragma unroll
          for (int e = 0; e < kEach; e += 2)
            *reinterpret_cast<uint32_t*>(a.o + out[k] * D + lane * kEach + e) = dev::pack_bf16(acc[k][e] * inv, acc[k][e + 1] * inv);
          if (lane == 0) a.lse[out[k]] = l[k] == 0.f ? -INFINITY : (m[k] + log2f(l[k])) * 0.69314718055994531f;
        }
    }
    return;
  }
  for (int r = blockIdx.y; r < P::kRows; r += gridDim.y) {
    int tok, head;
    if (!P::row(s, a.group, g.u, r, tok, head)) continue;
    // piece x is in block b's second slot or block b + x's first
    auto slot = [&](int x) { return static_cast<long long>(2 * (b + x) + (x == 0)) * P::kRows + r; };
    float m = -INFINITY;
    for (int x = tid; x < count; x += 32 * kMergeWarps) m = fmaxf(m, a.part_ml[slot(x)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) warp_ml[warp].x = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) m = fmaxf(m, warp_ml[w].x);
    const float mb = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    for (int x = tid; x < count; x += 32 * kMergeWarps) {
      const float2 ml = a.part_ml[slot(x)];
      const float f = exp2f(ml.x - mb);
      weight[x] = f;
      l = fmaf(f, ml.y, l);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) warp_ml[warp].y = l;
    __syncthreads();
    const int c = tid % kPieceLanes, x0 = tid / kPieceLanes;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int x = x0; x < count; x += kAtOnce) {
      const float4 y = reinterpret_cast<const float4*>(a.part_o + slot(x) * D)[c];
      const float f = weight[x];
      acc.x = fmaf(f, y.x, acc.x);
      acc.y = fmaf(f, y.y, acc.y);
      acc.z = fmaf(f, y.z, acc.z);
      acc.w = fmaf(f, y.w, acc.w);
    }
    part[x0][c] = acc;
    __syncthreads();
    if (tid < kPieceLanes) {
      l = 0.f;
#pragma unroll
      for (int w = 0; w < kMergeWarps; ++w) l += warp_ml[w].y;
#pragma unroll
      for (int x = 1; x < kAtOnce; ++x) {
        const float4 y = part[x][c];
        acc.x += y.x;
        acc.y += y.y;
        acc.z += y.z;
        acc.w += y.w;
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const long long row = static_cast<long long>(g.h * a.group + head) * a.c.total_new + s.a + tok;
      uint2 pk;
      pk.x = dev::pack_bf16(acc.x * inv, acc.y * inv);
      pk.y = dev::pack_bf16(acc.z * inv, acc.w * inv);
      reinterpret_cast<uint2*>(a.o + row * D)[c] = pk;
      if (c == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
    }
    __syncthreads();
  }
}

// Partial results, their statistics and the split groups' descriptors of a grid of up to
// `blocks` blocks.
inline size_t workspace_bytes(int rows, int d, int blocks) {
  return static_cast<size_t>(2 * blocks) * rows * (static_cast<size_t>(d) * sizeof(float) + sizeof(float2)) +
         blocks * sizeof(SplitGroup);
}
template <class P>
inline void set_workspace(AttnArgs& a, void* workspace, int d, int blocks) {
  const size_t rows = static_cast<size_t>(2 * blocks) * P::kRows;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + rows * d);
  a.split = reinterpret_cast<SplitGroup*>(a.part_ml + rows);
}

template <class P, int D>
inline fcp_status launch_merge(const AttnArgs& a, int blocks, int slices, cudaStream_t s) {
  return launch_overlapped(paged_merge_kernel<P, D>, dim3(blocks, slices), 32 * kMergeWarps, 0, s, "paged merge launch", a);
}

fcp_status launch_paged_few4(const AttnArgs& a, int d, int rows, void* workspace, int dev, int n_sm, int max_new,
                             cudaStream_t s);
fcp_status launch_paged_chunk(const AttnArgs& a, int dtype, int d, int hq, int max_new, void* workspace, int dev,
                              int n_sm, cudaStream_t s);

}  // namespace fcp
