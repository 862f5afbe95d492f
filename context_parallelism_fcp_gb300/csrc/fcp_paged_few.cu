// Attention of few new rows for each cached sequence (single tokens, drafted tokens) over a
// paged cache, and the entry point of the attention over a paged cache.
//
// For a KV head the rows are (new token, query head) pairs, 8, 16 or 32 to a unit, so every query
// head of the group and every drafted token shares one pass over the keys: HBM traffic is the
// cache once, at 4 * rows flops for every 2 bytes read: far below what the tensor cores need,
// so the kernel is bound by HBM and its business is to keep enough bytes in flight, and for an
// e4m3 cache to spend few enough instructions on a byte. Each warp takes every fourth 16-key
// chunk of its block's piece and runs its own pipeline of cp.async stages (a chunk lies in one
// page because pages are multiples of 16 keys) and its own running softmax; warps meet only at
// the end of a piece.
//
// The products are S^T = K Q^T and O^T += V^T P^T, m16n8k16 with float32 sums: keys and channels
// take the 16, rows the 8, so 8 rows (one token of 8 heads) fill the instruction, and K's and
// V's fragments serve all of a unit's rows. (With rows as the 16, half empty, 128 e4m3 sequences
// of up to 8192 keys took 171 us; tcgen05's 128 rows would be fifteen sixteenths empty.) A lane
// has two keys and two rows of S^T; movmatrix turns the weights into P^T's fragment.
//
// K is read from shared memory 16 bytes to a lane: the product over channels does not care for
// their order, so lane j of a quad takes 8 (bf16) or 16 (e4m3) neighbouring channels and Q's
// fragments are laid out the same way. V goes through ldmatrix.trans; for e4m3 the 16-bit
// elements that it transposes are channel pairs, whose low and high bytes become the two halves
// of a 16-channel fragment. 16-byte pieces of a row are XOR-swizzled so that neither reading has
// bank conflicts.
//
// An e4m3 cache's codes become f16 by the hardware's conversion, two to an instruction, and the
// products run in f16: a code is exact there, Q's rows are scaled to a largest exponent of 14
// (a power of two for each row, exact but for elements 2^-28 times the largest), and the rows'
// scales multiply the scores. V's scale goes into the exponent of P: with s' = s + log2(scale)
// the sum for O runs relative to the maximum of s', the sum of weights relative to that of s. A row of
// V whose scale is far below that of the keys with the large s' gets a P that f16 cannot hold: where
// a chunk has one, what f16 leaves of P is multiplied by V once more, scaled up.
//
// Measured (8 KV heads, D = 128): 128 e4m3 sequences of up to 8192 tokens, 8 query heads a KV head,
// 150 us (5870 GB/s, 87% of a copy's rate); two bf16 sequences of 131072, 155 us (6900 GB/s, all of
// it); 32 bf16 sequences of up to 4096 with 4 drafted tokens, 4 query heads a KV head, 39 us (5170
// GB/s, 76%; the beginnings and ends of pieces are the rest), and 38 us from an e4m3 cache, whose half
// as many bytes cost a conversion and two exponentials a weight (with 2 and 8 query heads a KV head 26.7
// and 57.6 us). 10 sequences of up to 1000 take 9 us, of which the lengths, the first rows and the merge
// are a dependent chain of memory latencies.
#include <algorithm>
#include <cmath>

#include "fcp_paged_sched.cuh"

namespace fcp {
namespace {

using namespace dev;

constexpr int kWarps = 4;
constexpr int kFewThreads = kWarps * 32;
constexpr int kChunk = 16;                  // keys of a stage
constexpr float kGrow = 8.0f;               // a row maximum is raised when it grows by over 2^8
constexpr float kUp = 7.0f;                 // e4m3: P starts at 2^7 and grows to 2^15, the top of f16
// e4m3: below 2^-14 P's rounding to f16 is off by up to 2^-25, which for a key whose V has a scale
// 2^gap below that of the largest is 2^(gap - 25 - kUp) of the largest weight. Up to this gap (2^-22)
// that is left so; beyond it the rest of P counts too (which it has to: with gaps of 2^18 and more,
// channels where the large row is zero were off by tens of times the rounding of P and o, or zero).
// The test for it costs single tokens up to 1%, 32 x 4 tokens of 2 and 4 heads 2%, of 8 nothing.
constexpr int kScaleGap = 10;
constexpr float kLift = 0x1p28f;
// Blocks to an SM and the shared memory of a block's stages, for NT tiles of 8 rows. bf16 is at
// HBM's rate with two; the e4m3 conversion leaves more latency to hide, as far as the registers
// go: 128, 168 and 255 a thread.
template <bool kE4M3, int NT>
constexpr int kPerSm = !kE4M3 ? 2 : (NT == 1 ? 4 : (NT == 2 ? 3 : 2));

template <int D, bool kE4M3, int NT>
struct FewCfg {
  static constexpr int kStageBudget = (kPerSm<kE4M3, NT> == 4 ? 50 : (kPerSm<kE4M3, NT> == 3 ? 67 : 97)) * 1024;
  static constexpr int kRowBytes = kE4M3 ? D : 2 * D;
  static constexpr int kPieces = kRowBytes / 16;               // 16-byte pieces of a row
  static constexpr int kTile = kChunk * kRowBytes;             // K or V of a chunk
  static constexpr int kStage = 2 * kTile + (kE4M3 ? 32 : 0);  // + 16 K scales, 16 V scales
  static constexpr int kStagesRaw = kStageBudget / (kWarps * kStage);
  static constexpr int kStages = kStagesRaw > 8 ? 8 : kStagesRaw;
  static constexpr int kWarpBytes = kStages * kStage;
};

// Where piece c of row r lies in a tile. Rows of 128 bytes and more: 8 rows of one piece, and
// pieces 0-3 of two neighbouring rows, fall on different banks; rows of 64 bytes share a line
// of banks two by two.
template <int kRowBytes>
__device__ __forceinline__ int piece_at(int r, int c) {
  if constexpr (kRowBytes == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  else return r * kRowBytes + ((c ^ (((r & 1) << 2) | ((r >> 1) & 3))) << 4);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16_or_zeros(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// c[16 x 8] += a[16 x 16] b[16 x 8], bf16 in, float32 out
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// the same in f16
__device__ __forceinline__ void mma16816h(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The 8x8 matrix of 16-bit elements that the warp holds, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// f(c, fragment) for each 16 channels of a chunk's V in e4m3, as the first operand in f16.
template <int kRowBytes, class F>
__device__ __forceinline__ void each_v(uint32_t vt, int lane, F f) {
  const int vr = (lane & 7) + (lane & 8);  // keys 0-7, 8-15 of a 16-channel piece, then of the next
#pragma unroll
  for (int c = 0; c < kRowBytes / 16; c += 2) {
    uint32_t x[4];
    ldsm4_trans(vt + piece_at<kRowBytes>(vr, c + (lane >> 4)), x);
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      // bytes: even and odd channel of one key, then of the next; the even channels are the
      // fragment's rows 0-7, the odd ones 8-15
      uint32_t v[4];
      e4m3x4_to_f16x2(__byte_perm(x[2 * y], 0, 0x3120), v[0], v[1]);
      e4m3x4_to_f16x2(__byte_perm(x[2 * y + 1], 0, 0x3120), v[2], v[3]);
      f(c + y, v);
    }
  }
}

struct Piece {
  int valid, i, h, u, a, n, len, end, ga, gb, slot;
};

template <int D, bool kE4M3, int NT>
__global__ void __launch_bounds__(kFewThreads, kPerSm<kE4M3, NT>) few_kernel(const AttnArgs a) {
  using C = FewCfg<D, kE4M3, NT>;
  using P = FewRows<8 * NT>;
  constexpr int kRows = P::kRows;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Line<kFewThreads> line;
  __shared__ Walk<P> walk;
  __shared__ Piece shared_piece[2];  // the one at work, and the next
  __shared__ float warp_m[kWarps][kRows], warp_l[kWarps][kRows];
  __shared__ uint2 shared_q[NT == 4 ? NT : 1][NT == 4 ? D / 16 : 1][32];
  __shared__ float shared_back[32];
  static_assert(NT != 4 || NT == kWarps, "a warp prepares each tile of Q");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // this lane's fragment row (a key, or a channel; and that + 8) and its pair of columns
  const int i8 = lane >> 2, j = lane & 3;
  const int b = blockIdx.x;
  let_next_start();
  wait_for_previous();
  if (threadIdx.x == 0) a.split[b].last = b;
  const uint32_t stages = smem_u32(smem) + warp * C::kWarpBytes;
  // [kWarps][kRows][kSumRow], over the stages at a piece's end; 4 floats between rows keep a warp's
  // stores on different banks
  float* sums = reinterpret_cast<float*>(smem);
  constexpr int kSumRow = D + 4;
  static_assert(kWarps * kRows * kSumRow * 4 <= C::kStageBudget, "the warps' sums fit the stages");
  const int page_mask = (1 << a.c.page_shift) - 1;

  // One thread walks on to the share's next piece, w1 being the share's end.
  auto advance = [&](Walk<P>& w, const Shares& sh, long long w0, long long w1, Piece& to) {
    Piece p;
    p.ga = p.gb = 0;
    while ((p.valid = w.i < a.c.n_seqs && w.f0 < w1)) {
      w.part(w0, w1, p.ga, p.gb);
      if (p.gb > p.ga) break;
      w.next(a, line, w1);  // the share has the group's overhead only
    }
    if (p.valid) {
      p.i = w.i;
      p.h = w.h;
      p.u = w.u;
      p.a = w.s.a;
      p.n = w.s.n;
      p.len = w.s.len;
      p.end = w.end;
      p.slot = piece_slot(b, p.ga, p.gb, w.g);
      if (p.ga == 0 && p.gb < w.g) a.split[b] = SplitGroup{sh.owner(w.behind() - 1), w.s.a, w.s.n, w.h, w.u, {}};
    }
    walk = w;
    to = p;
  };
  const Shares sh = begin_walk<P, kFewThreads>(a, line, b == 0, [&](Walk<P>& w, const Shares& sh, long long w0, long long w1) {
    advance(w, sh, w0, w1, shared_piece[0]);
  });
  if (b >= sh.blocks) return;
  // Chunks of this warp are keys k0 + 16 * (warp + 4 n) below kend. Lane l holds the block table's
  // entry for chunk l of a batch of 32.
  auto entries = [&](const Piece& p, int batch) -> int {
    const int key = p.ga * kGranule + kChunk * (warp + kWarps * (32 * batch + lane));
    return p.valid && key < min(p.gb * kGranule, p.end)
               ? load(a.c.table + static_cast<long long>(p.i) * a.c.max_pages + (key >> a.c.page_shift))
               : -1;
  };
  int pages = entries(shared_piece[0], 0);
  for (int turn = 0;; turn ^= 1) {
    const Piece p = shared_piece[turn];
    if (!p.valid) break;
    const SeqShape s{p.a, p.n, p.len};
    const int k0 = p.ga * kGranule, kend = min(p.gb * kGranule, p.end);
    const int key0 = k0 + kChunk * warp;
    int pages_next = entries(p, 1);
    // (token, head of the group) of the unit's row r, which lane r works out
    int my_tok, my_head;
    P::row(s, a.group, p.u, lane & (kRows - 1), my_tok, my_head);
    auto row = [&](int r, int& tok, int& head) -> bool {
      tok = __shfl_sync(0xffffffffu, my_tok, r);
      head = __shfl_sync(0xffffffffu, my_head, r);
      return tok < s.n;
    };

    // Q as the second operand: tile t's row 8 t + i8. With four tiles it would take a quarter of the
    // registers: warp t prepares tile t, and all read it from shared memory.
    constexpr bool kSharedQ = NT == 4;
    uint32_t q[kSharedQ ? 1 : NT][D / 16][2];
#pragma unroll
    for (int t = 0; t < (kSharedQ ? 1 : NT); ++t) {
      int tok, head;
      const bool on = row(8 * (kSharedQ ? warp : t) + i8, tok, head);
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + (static_cast<long long>(p.h * a.group + (on ? head : 0)) * a.c.total_new + s.a + (on ? tok : 0)) * D);
      if constexpr (kE4M3) {
        // 64 channels: lane j has channels 16 j .. 16 j + 15, in products 0-3 of the 64
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint4 v = on ? load(src + c * 8 + 2 * j + y) : make_uint4(0, 0, 0, 0);
            q[t][4 * c + 2 * y][0] = v.x;
            q[t][4 * c + 2 * y][1] = v.y;
            q[t][4 * c + 2 * y + 1][0] = v.z;
            q[t][4 * c + 2 * y + 1][1] = v.w;
          }
      } else {
        // 32 channels: lane j has channels 8 j .. 8 j + 7, in products 0-1 of the 32
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          const uint4 v = on ? load(src + c * 4 + j) : make_uint4(0, 0, 0, 0);
          q[t][2 * c][0] = v.x;
          q[t][2 * c][1] = v.y;
          q[t][2 * c + 1][0] = v.z;
          q[t][2 * c + 1][1] = v.w;
        }
      }
    }

    int n_issued = 0, issue_stage = 0;
    auto issue = [&]() {
      const int key = key0 + n_issued * (kChunk * kWarps);
      if (key < kend) {
        if ((n_issued & 31) == 0 && n_issued > 0) {
          pages = pages_next;
          pages_next = entries(p, (n_issued >> 5) + 1);
        }
        const int page = __shfl_sync(0xffffffffu, pages, n_issued & 31);
        const bool ok = static_cast<unsigned>(page) < static_cast<unsigned>(a.c.n_pages);
        if (!ok && lane == 0) atomicCAS(a.c.status, 0, kErrCachePage);
        const long long r0 = ok ? page_row(a.c, page, p.h) + (key & page_mask) : 0;
        const uint32_t dst = stages + issue_stage * C::kStage;
        constexpr int kPer = 32 / C::kPieces;  // rows of one instruction
        const int lr = lane / C::kPieces, c = lane % C::kPieces;
        const long long at = (r0 + lr) * C::kRowBytes + c * 16;
        const uint8_t* gk = a.c.k_pages + at;
        const uint8_t* gv = a.c.v_pages + at;
        if (ok && key + kChunk <= s.len) {
#pragma unroll
          for (int x = 0; x < kChunk / kPer; ++x) {
            const int to = piece_at<C::kRowBytes>(x * kPer + lr, c);
            cp_async16(dst + to, gk + x * kPer * C::kRowBytes);
            cp_async16(dst + C::kTile + to, gv + x * kPer * C::kRowBytes);
          }
        } else {  // rows behind the last key may hold anything: zeros come in their place
#pragma unroll 1
          for (int x = 0; x < kChunk / kPer; ++x) {
            const bool on = ok && key + x * kPer + lr < s.len;
            const int to = piece_at<C::kRowBytes>(x * kPer + lr, c);
            cp_async16_or_zeros(dst + to, on ? gk + x * kPer * C::kRowBytes : a.c.k_pages, on);
            cp_async16_or_zeros(dst + C::kTile + to, on ? gv + x * kPer * C::kRowBytes : a.c.v_pages, on);
          }
        }
        if constexpr (kE4M3) {
          if (lane < 2)
            cp_async16_or_zeros(dst + 2 * C::kTile + 16 * lane, (lane ? a.c.v_scales : a.c.k_scales) + r0, ok);
        }
      }
      cp_commit();
      ++n_issued;
      issue_stage = issue_stage + 1 == C::kStages ? 0 : issue_stage + 1;
    };
#pragma unroll
    for (int x = 0; x < C::kStages - 1; ++x) issue();
    // while Q and the first chunks are on their way, in the warp that has the fewest
    if (threadIdx.x == kFewThreads - 32) {
      Walk<P> w = walk;
      const long long w1 = sh.begin(b + 1);
      w.next(a, line, w1);
      advance(w, sh, sh.begin(b), w1, shared_piece[turn ^ 1]);
    }

    // e4m3: Q's rows as f16 scaled by 2^(14 - e), e the largest exponent of the row; `back` takes the
    // scores of row i8 of a tile to log2 units.
    float back[kSharedQ ? 1 : NT];
#pragma unroll
    for (int t = 0; t < (kSharedQ ? 1 : NT); ++t) {
      back[t] = a.scale_log2;
      if constexpr (kE4M3) {
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
#pragma unroll
          for (int y = 0; y < 2; ++y) top = max(top, max(q[t][c][y] & 0x7fffu, (q[t][c][y] >> 16) & 0x7fffu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int up = min(126, 141 - static_cast<int>(top >> 7));  // 14 - (exponent - 127), of rows past 2^-112
        const float f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
#pragma unroll
          for (int y = 0; y < 2; ++y)
            q[t][c][y] = pack_f16(__uint_as_float(q[t][c][y] << 16) * f, __uint_as_float(q[t][c][y] & 0xffff0000u) * f);
        back[t] *= __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
      }
    }
    if constexpr (kSharedQ) {
#pragma unroll
      for (int c = 0; c < D / 16; ++c) shared_q[warp][c][lane] = make_uint2(q[0][c][0], q[0][c][1]);
      if (j == 0) shared_back[8 * warp + i8] = back[0];
      __syncthreads();
    }
    // first key that some row does not see
    const int lim_min = a.causal ? s.len - s.n + __shfl_sync(0xffffffffu, my_tok, 0) + 1 : s.len;
    // The lane's columns of S^T are rows 8 t + 2 j + {0, 1}: the first key that each does not see, and
    // its factor.
    int lim[NT][2];
    float factor[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        int tok, head;
        const bool on = row(8 * t + 2 * j + e, tok, head);
        lim[t][e] = !on || !a.causal ? s.len : s.len - s.n + tok + 1;
        if constexpr (kSharedQ) factor[t][e] = shared_back[8 * t + 2 * j + e];
        else factor[t][e] = kE4M3 ? __shfl_sync(0xffffffffu, back[t], 4 * (2 * j + e)) : a.scale_log2;
      }
    auto q_of = [&](int t, int c) -> uint2 {
      if constexpr (kSharedQ) return shared_q[t][c][lane];
      else return make_uint2(q[t][c][0], q[t][c][1]);
    };

    // m: the maximum of a row's scores, which its weights' sum l is relative to; mo: for e4m3 that of
    // scores with V's scale less kUp, which acc is relative to. The eight lanes of a column pair share m
    // and mo; l is over the lane's own keys. low: the scale byte below which a row of V is far below mo.
    int low = 0;
    float m[NT][2], l[NT][2], mo[NT][2], acc[D / 16][NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[t][e] = mo[t][e] = -INFINITY;
        l[t][e] = 0.f;
      }
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[c][t][e] = 0.f;
    }

    int stage = 0;
    for (int key = k0 + kChunk * warp; key < kend; key += kChunk * kWarps) {
      cp_wait<C::kStages - 2>();
      __syncwarp();  // this chunk has arrived, and every lane is done with the stage that is filled next
      issue();
      const uint32_t kt = stages + stage * C::kStage, vt = kt + C::kTile;
      stage = stage + 1 == C::kStages ? 0 : stage + 1;

      // S^T: element 2 y + e is key + 8 y + i8, row 8 t + 2 j + e
      float sc[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[t][e] = 0.f;
      if constexpr (kE4M3) {
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const uint4 v0 = lds16(kt + piece_at<C::kRowBytes>(i8, 4 * c + j));
          const uint4 v1 = lds16(kt + piece_at<C::kRowBytes>(8 + i8, 4 * c + j));
          const uint32_t raw0[4] = {v0.x, v0.y, v0.z, v0.w}, raw1[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t f[4];
            e4m3x4_to_f16x2(raw0[x], f[0], f[2]);
            e4m3x4_to_f16x2(raw1[x], f[1], f[3]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const uint2 y = q_of(t, 4 * c + x);
              mma16816h(sc[t], f, y.x, y.y);
            }
          }
        }
      } else {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          const uint4 v0 = lds16(kt + piece_at<C::kRowBytes>(i8, 4 * c + j));
          const uint4 v1 = lds16(kt + piece_at<C::kRowBytes>(8 + i8, 4 * c + j));
          const uint32_t lo[4] = {v0.x, v1.x, v0.y, v1.y}, hi[4] = {v0.z, v1.z, v0.w, v1.w};
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const uint2 y0 = q_of(t, 2 * c), y1 = q_of(t, 2 * c + 1);
            mma16816(sc[t], lo, y0.x, y0.y);
            mma16816(sc[t], hi, y1.x, y1.y);
          }
        }
      }
      // Scores in log2 units; for e4m3 `so` is the score with log2 of V's scale added. Lane l turns one
      // of the 32 scales (16 of K, 16 of V) into what is needed of it, and the others ask for it.
      float so[NT][4];
      float kf[2], vf[2];
      uint32_t byte = 0;
      if constexpr (kE4M3) {
        byte = lds_u8(kt + 2 * C::kTile + lane);
        const float mine = lane < 16 ? e8m0_to_float(byte) : e8m0_log2(byte);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          kf[y] = __shfl_sync(0xffffffffu, mine, 8 * y + i8);
          vf[y] = __shfl_sync(0xffffffffu, mine, 16 + 8 * y + i8);
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (kE4M3) {
            sc[t][e] *= factor[t][e & 1] * kf[e >> 1];
            so[t][e] = sc[t][e] + vf[e >> 1];
          } else {
            sc[t][e] *= factor[t][e & 1];
          }
        }
      if (key + kChunk > lim_min) {  // some row does not see the whole chunk
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (key + 8 * (e >> 1) + i8 >= lim[t][e & 1]) sc[t][e] = so[t][e] = -INFINITY;
      }
      // raise the running maxima only when some row's grew by more than 2^8: P stays below 2^8
      bool grow = false;
      float top[NT][2], topo[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[t][e] = fmaxf(sc[t][e], sc[t][2 + e]);
          grow = grow || top[t][e] > m[t][e] + kGrow;
          if constexpr (kE4M3) {
            topo[t][e] = fmaxf(so[t][e], so[t][2 + e]);
            grow = grow || topo[t][e] > mo[t][e] + (kGrow + kUp);
          }
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            auto raise = [](float& at, float to) -> float {  // the factor of what was relative to `at`
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, o));
              to = fmaxf(to, at);
              const float f = to == -INFINITY ? 1.f : fast_exp2(at - to);
              at = to;
              return f;
            };
            float f = raise(m[t][e], top[t][e]);
            l[t][e] *= f;
            if constexpr (kE4M3) f = raise(mo[t][e], topo[t][e] - kUp);
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              acc[c][t][e] *= f;
              acc[c][t][2 + e] *= f;
            }
          }
        if constexpr (kE4M3) {
          float gap = -INFINITY;
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) gap = fmaxf(gap, mo[t][e] - m[t][e]);  // rows without a key: NaN, left out
#pragma unroll
          for (int o = 1; o < 4; o <<= 1) gap = fmaxf(gap, __shfl_xor_sync(0xffffffffu, gap, o));
          low = lane < 16 ? 0 : static_cast<int>(fmaxf(gap, -256.f) + kUp) + 127 - kScaleGap;
        }
      }
      // P^T: the packed pairs are (key; rows 2 j, 2 j + 1) and are wanted as (row; keys 2 j, 2 j + 1)
      uint32_t pt[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float pw[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          pw[e] = fast_exp2(sc[t][e] - (m[t][e & 1] == -INFINITY ? 0.f : m[t][e & 1]));
          l[t][e & 1] += pw[e];
          // in f16: off by 2^-11 of itself, or 2^-25 (see kScaleGap)
          if constexpr (kE4M3) pw[e] = fast_exp2(so[t][e] - (mo[t][e & 1] == -INFINITY ? 0.f : mo[t][e & 1]));
        }
#pragma unroll
        for (int y = 0; y < 2; ++y)
          pt[t][y] = transpose8x8(kE4M3 ? pack_f16(pw[2 * y], pw[2 * y + 1])
                                        : pack_bf16(pw[2 * y], pw[2 * y + 1]));  // bf16: off by 2^-8 of itself at most
      }
      if constexpr (kE4M3) {
        if (__any_sync(0xffffffffu, static_cast<int>(byte) < low)) {  // of V's scales: lanes 16 and on
          // What is left of P where f16 rounds it as a subnormal number, times 2^28, then what is left of
          // that: each product's sum is added at its own scale. (A tile of rows at a time, for registers.)
          auto left = [](float x) -> float {
            return fabsf(x) < 0x1p-14f ? (x - __half2float(__float2half_rn(x))) * kLift : 0.f;
          };
#pragma unroll
          for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int e = 0; e < 4; ++e) so[t][e] = left(fast_exp2(so[t][e] - (mo[t][e & 1] == -INFINITY ? 0.f : mo[t][e & 1])));
            float down = 1.f;
#pragma unroll 1
            while (__any_sync(0xffffffffu, so[t][0] != 0.f || so[t][1] != 0.f || so[t][2] != 0.f || so[t][3] != 0.f)) {
              uint32_t rest[2];
#pragma unroll
              for (int y = 0; y < 2; ++y) rest[y] = transpose8x8(pack_f16(so[t][2 * y], so[t][2 * y + 1]));
#pragma unroll
              for (int e = 0; e < 4; ++e) so[t][e] = left(so[t][e]);
              down *= 1.f / kLift;
              each_v<C::kRowBytes>(vt, lane, [&](int c, const uint32_t(&v)[4]) {
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
                mma16816h(sum, v, rest[0], rest[1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[c][t][e] = fmaf(sum[e], down, acc[c][t][e]);
              });
            }
          }
        }
      }
      if constexpr (kE4M3) {
        each_v<C::kRowBytes>(vt, lane, [&](int c, const uint32_t(&v)[4]) {
#pragma unroll
          for (int t = 0; t < NT; ++t) mma16816h(acc[c][t], v, pt[t][0], pt[t][1]);
        });
      } else {
        const int vr = (lane & 7) + ((lane >> 4) << 3);  // channels 0-7, 8-15 of keys 0-7, then of keys 8-15
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          uint32_t v[4];
          ldsm4_trans(vt + piece_at<C::kRowBytes>(vr, 2 * c + ((lane >> 3) & 1)), v);
#pragma unroll
          for (int t = 0; t < NT; ++t) mma16816(acc[c][t], v, pt[t][0], pt[t][1]);
        }
      }
    }
    cp_wait<0>();

    // the warps' sums meet: every row relative to the largest of the warps' maxima
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], o);
        if (i8 == 0) warp_m[warp][8 * t + 2 * j + e] = m[t][e];
      }
    __syncthreads();  // also: every warp is done with its stages, and the next piece is there
    pages = entries(shared_piece[turn ^ 1], 0);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * t + 2 * j + e;
        float mx = warp_m[0][r];
#pragma unroll
        for (int y = 1; y < kWarps; ++y) mx = fmaxf(mx, warp_m[y][r]);
        float f = mx == -INFINITY ? 0.f : fast_exp2(m[t][e] - mx);
        if (i8 == 0) warp_l[warp][r] = l[t][e] * f;
        if constexpr (kE4M3) f = mx == -INFINITY ? 0.f : fast_exp2(mo[t][e] - mx);  // acc's own reference
        float* dst = sums + (static_cast<size_t>(warp) * kRows + r) * kSumRow;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const float x0 = acc[c][t][e] * f, x1 = acc[c][t][2 + e] * f;
          if constexpr (kE4M3) {  // channels 2 i8 and 2 i8 + 1 of the 16
            *reinterpret_cast<float2*>(dst + 16 * c + 2 * i8) = make_float2(x0, x1);
          } else {
            dst[16 * c + i8] = x0;
            dst[16 * c + 8 + i8] = x1;
          }
        }
      }
    __syncthreads();
    constexpr int kLanes = D / 4;
    for (int x = threadIdx.x; x < kRows * kLanes; x += kFewThreads) {
      const int r = x / kLanes, c = x % kLanes;
      int tok, head;
      if (!row(r, tok, head)) continue;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      float sum = 0.f, mx = -INFINITY;
#pragma unroll
      for (int y = 0; y < kWarps; ++y) {
        const float4 v = reinterpret_cast<const float4*>(sums + (static_cast<size_t>(y) * kRows + r) * kSumRow)[c];
        o.x += v.x;
        o.y += v.y;
        o.z += v.z;
        o.w += v.w;
        sum += warp_l[y][r];
        mx = fmaxf(mx, warp_m[y][r]);
      }
      if (p.slot < 0) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const long long at = static_cast<long long>(p.h * a.group + head) * a.c.total_new + s.a + tok;
        uint2 pk;
        pk.x = pack_bf16(o.x * inv, o.y * inv);
        pk.y = pack_bf16(o.z * inv, o.w * inv);
        reinterpret_cast<uint2*>(a.o + at * D)[c] = pk;
        if (c == 0) a.lse[at] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * 0.69314718055994531f;
      } else {
        const long long at = static_cast<long long>(p.slot) * kRows + r;
        reinterpret_cast<float4*>(a.part_o + at * D)[c] = o;
        if (c == 0) a.part_ml[at] = make_float2(mx, sum);
      }
    }
    __syncthreads();  // the stages are free again
  }
}

template <int D, bool kE4M3, int NT>
fcp_status launch_few(AttnArgs a, void* workspace, int dev, int n_sm, int max_new, cudaStream_t s) {
  using C = FewCfg<D, kE4M3, NT>;
  using P = FewRows<8 * NT>;
  constexpr int kSmem = std::max(kWarps * C::kWarpBytes, kWarps * P::kRows * (D + 4) * 4);
  const int blocks = std::min(kPerSm<kE4M3, NT> * n_sm, kMaxBlocks);
  set_workspace<P>(a, workspace, D, kMaxBlocks);
  static std::atomic<uint64_t> allowed{0};
  if (const fcp_status st = allow_smem(few_kernel<D, kE4M3, NT>, kSmem, dev, allowed, "paged attention smem attribute");
      st != FCP_OK)
    return st;
  if (const fcp_status st = launch_overlapped(few_kernel<D, kE4M3, NT>, dim3(blocks), kFewThreads, kSmem, s,
                                              "paged attention launch", a);
      st != FCP_OK)
    return st;
  // the merge's row slices: a warp takes two rows where groups have few pieces (many groups), else a
  // block takes one
  const long long rows = std::min<long long>(static_cast<long long>(std::max(max_new, 1)) * a.group, P::kRows);
  const bool few_pieces = static_cast<long long>(P::kWarpPieces) * a.c.n_seqs * a.c.hkv >= blocks;
  return launch_merge<P, D>(
      a, blocks, static_cast<int>(few_pieces ? (rows + 2 * kMergeWarps - 1) / (2 * kMergeWarps) : rows), s);
}

template <int D>
fcp_status launch_attn(const AttnArgs& a, int dtype, int hq, int max_new, void* workspace, cudaStream_t s) {
  int dev = 0, n_sm = 0;
  if (const fcp_status st = this_device(&dev, &n_sm); st != FCP_OK) return st;
  const long long rows = static_cast<long long>(max_new) * a.group;
  // Up to 32 rows of a KV head this kernel, in as few tiles of 8 as hold them; beyond, the tensor
  // core's tiles of 128. (With 64 rows as the border, in two units: 48 rows took 19.0 us instead of
  // 20.8 from an e4m3 cache and 16.6 instead of 19.6 from a bf16 one, 60 rows 21.4 instead of 18.5,
  // 64 rows of long sequences 37.4 instead of 36.7, 128 rows far more.)
  if (rows > 32) return launch_paged_chunk(a, dtype, D, hq, workspace, dev, n_sm, s);
  const bool e = dtype == FCP_CACHE_E4M3;
  auto* launch = rows <= 8    ? (e ? launch_few<D, true, 1> : launch_few<D, false, 1>)
                 : rows <= 16 ? (e ? launch_few<D, true, 2> : launch_few<D, false, 2>)
                              : (e ? launch_few<D, true, 4> : launch_few<D, false, 4>);
  return launch(a, workspace, dev, n_sm, max_new, s);
}

}  // namespace
}  // namespace fcp

using namespace fcp;

extern "C" size_t fcp_paged_attn_workspace_bytes(int32_t head_dim) {
  if (head_dim != 64 && head_dim != 128) return 0;
  return std::max(workspace_bytes(ChunkRows::kRows, head_dim, kMaxChunkBlocks), workspace_bytes(32, head_dim, kMaxBlocks));
}

extern "C" fcp_status fcp_paged_attn(const fcp_cache* cache, const fcp_cache_batch* batch, const void* q, int32_t hq,
                                     int32_t causal, void* o, float* lse, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  AttnArgs a;
  if (const fcp_status st = paged_args(cache, batch, &a.c); st != FCP_OK) return st;
  if (hq <= 0 || hq % cache->hkv != 0) return FCP_ERR_INVALID;
  if (a.c.total_new == 0 || a.c.n_seqs == 0) return FCP_OK;
  if (!q || !o || !lse || !workspace || !aligned16(q) || !aligned16(o) || !aligned4(lse) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return FCP_ERR_INVALID;
  if (workspace_bytes < fcp_paged_attn_workspace_bytes(cache->head_dim)) return FCP_ERR_INVALID;
  a.group = hq / cache->hkv;
  a.causal = causal ? 1 : 0;
  a.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(cache->head_dim)));
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.small = (static_cast<long long>(a.c.max_pages) << a.c.page_shift) * a.c.n_seqs * cache->hkv <= 1 << 18;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cache->head_dim == 128 ? launch_attn<128>(a, cache->dtype, hq, batch->max_new, workspace, s)
                                : launch_attn<64>(a, cache->dtype, hq, batch->max_new, workspace, s);
}
