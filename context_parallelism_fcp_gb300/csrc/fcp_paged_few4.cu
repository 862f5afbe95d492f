// Attention of few new rows for each cached sequence over a paged cache in 4 bits.
//
// As the kernels of fcp_paged_few.cu (rows of a KV head share one pass over the keys; S^T = K Q^T and
// O^T += V^T P^T with keys and channels as the instruction's 16 and rows as its 8; every warp with its own
// cp.async pipeline and running softmax), with a cache of a quarter of bf16's bytes, so that the
// instructions spent on a code decide. e2m1 codes become f16 by the hardware's conversion, two to an
// instruction, and a multiplication by the e4m3 scale of their 16 channels, both exact; Q's rows are
// scaled to a largest exponent of 14, and P to 2^7 and up, so that f16 holds what counts of both.
//
// K's product over channels does not care for their order: lane j of a quad reads D / 4 neighbouring
// channels of a key. V goes through ldmatrix.trans as 16-bit elements of four channels: a register
// then has those of two keys, in its halves, and byte permutations put the same channel of both side by
// side, as the product over keys wants them.
//
// Measured (8 KV heads, D = 128): 128 sequences of up to 8192 tokens, 8 query heads a KV head, 103 us (4970
// GB/s, 74% of a copy's rate); of up to 32768, 348 us (87%): some 20 us are launch, merge and the beginnings and
// ends of three pieces a block. 32 sequences of up to 4096 with 4 drafted tokens and 2, 4, 8 query heads a KV
// head: 24.2, 28.6, 43.0 us. Issue slots 60% busy, the unit that converts and permutes 58%; with the
// conversions of codes taken out the first case took 105.6 instead of 108.8 us (then), so it is the sum of
// instructions and latencies at 12 warps an SM, not one of them. Not faster: copies that run on into the next
// piece (106), codes put side by side by logic before the conversion (111 instead of 108.5), one chunk a
// stage (114 instead of 108.5).
#include <algorithm>

#include "fcp_paged_few.cuh"

namespace fcp {
namespace {

using namespace dev;
using namespace few;

// Blocks to an SM: more registers are worth more than more warps (one tile: 128 sequences of up to 8192 103 us
// with three, 108 with four, of up to 32768 349 and 371; two tiles, 32 x 4 tokens: 28.9 with two, 30.4 with
// three, but 21.2 and 20.3 at D = 64).
template <int NT>
constexpr int kPerSm = NT == 1 ? 3 : 2;
// A piece's beginning and end are as long on the line as 3 granules: with 1, 2, 3, 5 the first case took 107.4,
// 104.2, 103.2, 104.9 us, 32 x 4 tokens of 8 heads 59.9, 46.4, 44.6, 47.6.
template <int NT>
using Rows = FewRows<8 * NT, 3>;

template <int D, int NT>
struct Cfg {
  static constexpr int kBudget = (kPerSm<NT> == 3 ? 67 : 97) * 1024;  // of shared memory
  static constexpr int kRowBytes = D / 2, kScales = D / 16;  // of a row of K or V
  static constexpr int kPieces = kRowBytes / 16;             // 16-byte pieces of a row
  // A stage is two chunks, whose overhead is shared and which are done together, for more independent
  // instructions.
  static constexpr int kKeys = 2 * kChunk;
  static constexpr int kTile = kKeys * kRowBytes;                  // K or V of a stage
  static constexpr int kScaleTile = kKeys * kScales;
  static constexpr int kStage = 2 * (kTile + kScaleTile);          // K, V, their scales
  static constexpr int kStages = std::min(8, kBudget / (kWarps * kStage));
  static constexpr int kWarpBytes = kStages * kStage;
  static_assert(kStages >= 2, "one stage on its way while one is at work");
};

__device__ __forceinline__ uint2 lds8(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds4(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
  uint32_t v;
  asm volatile("{\n.reg .b16 h;\nld.shared.b16 h, [%1];\ncvt.u32.u16 %0, h;\n}" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// The first `bytes` of 16, and zeros.
__device__ __forceinline__ void cp_async16_part(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// One half of a register, twice.
__device__ __forceinline__ uint32_t half_of(uint32_t x, int high) {
  const __half2 h = *reinterpret_cast<const __half2*>(&x), r = high ? __high2half2(h) : __low2half2(h);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Four codes of each of two keys (the low and the high half), times the keys' scales: the same code of
// both keys in one register.
__device__ __forceinline__ void pairs(uint32_t x, uint32_t scale, uint32_t (&r)[4]) {
  uint32_t h[4];
  e2m1x8_to_f16x2(x, h);
  r[0] = mul_f16x2(__byte_perm(h[0], h[2], 0x5410), scale);
  r[1] = mul_f16x2(__byte_perm(h[0], h[2], 0x7632), scale);
  r[2] = mul_f16x2(__byte_perm(h[1], h[3], 0x5410), scale);
  r[3] = mul_f16x2(__byte_perm(h[1], h[3], 0x7632), scale);
}

// f(c, fragment) for each 16 channels of a chunk's V, as the first operand: lane (i8, j) has channels
// 32 (c / 2) + 4 i8 + 2 (c % 2) and the next, as the fragment's rows i8 and 8 + i8.
template <int D, class F>
__device__ __forceinline__ void each_v(uint32_t vt, uint32_t scales, int lane, F f) {
  constexpr int kRowBytes = D / 2, kSegments = D / 32;
  const int vr = (lane & 7) + (lane & 8), j = lane & 3;
  const bool odd = (lane >> 4) != 0;  // channels 16-31 of a segment of 32
  uint32_t sc[2][kSegments];          // scales of keys 2 j and 2 j + 1 (and those + 8)
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const uint32_t at = scales + (8 * y + 2 * j) * (D / 16);
    if constexpr (D == 128) {
      const uint4 w = lds16(at);
      const uint32_t sel = odd ? 0x7531u : 0x6420u;
      const uint32_t k0 = __byte_perm(w.x, w.y, sel), k1 = __byte_perm(w.z, w.w, sel);
      e4m3x4_to_f16x2(__byte_perm(k0, k1, 0x5140), sc[y][0], sc[y][1]);
      e4m3x4_to_f16x2(__byte_perm(k0, k1, 0x7362), sc[y][2], sc[y][3]);
    } else {
      const uint2 w = lds8(at);
      e4m3x4_to_f16x2(__byte_perm(w.x, w.y, odd ? 0x7351u : 0x6240u), sc[y][0], sc[y][1]);
    }
  }
#pragma unroll
  for (int g = 0; g < kSegments; g += 2) {
    uint32_t x[4];
    ldsm4_trans(vt + piece_at<kRowBytes>(vr, g + (lane >> 4)), x);
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      uint32_t lo[4], hi[4];
      pairs(x[2 * y], sc[0][g + y], lo);
      pairs(x[2 * y + 1], sc[1][g + y], hi);
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const uint32_t v[4] = {lo[2 * z], lo[2 * z + 1], hi[2 * z], hi[2 * z + 1]};
        f(2 * (g + y) + z, v);
      }
    }
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(kFewThreads, kPerSm<NT>) few4_kernel(const AttnArgs a) {
  using C = Cfg<D, NT>;
  using P = Rows<NT>;
  constexpr int kRows = P::kRows, kKeys = C::kKeys;
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
  static_assert(kWarps * kRows * kSumRow * 4 <= C::kBudget, "the warps' sums fit the stages");
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
  // Stage n of this warp has keys k0 + kKeys * (warp + 4 n) and on, below kend. Lane l holds the block
  // table's entry for chunk l of a batch of 16 stages.
  auto entries = [&](const Piece& p, int batch) -> int {
    const int key = p.ga * kGranule + kKeys * (warp + kWarps * (16 * batch + (lane >> 1))) + kChunk * (lane & 1);
    return p.valid && key < min(p.gb * kGranule, p.end)
               ? load(a.c.table + static_cast<long long>(p.i) * a.c.max_pages + (key >> a.c.page_shift))
               : -1;
  };
  // Which 16 bytes of a stage's scales this lane copies: of K's two chunks, then of V's.
  constexpr int kScalePieces = C::kScaleTile / 16;
  const bool scales_of_v = lane >= kScalePieces;
  const int scale_chunk = lane % kScalePieces / (kScalePieces / 2), scale_at = 16 * (lane % (kScalePieces / 2));
  int pages = entries(shared_piece[0], 0);
  for (int turn = 0;; turn ^= 1) {
    const Piece p = shared_piece[turn];
    if (!p.valid) break;
    const SeqShape s{p.a, p.n, p.len};
    const int k0 = p.ga * kGranule, kend = min(p.gb * kGranule, p.end);
    const int key0 = k0 + kKeys * warp;
    int pages_next = entries(p, 1);
    // (token, head of the group) of the unit's row r, which lane r works out
    int my_tok, my_head;
    P::row(s, a.group, p.u, lane & (kRows - 1), my_tok, my_head);
    auto row = [&](int r, int& tok, int& head) -> bool {
      tok = __shfl_sync(0xffffffffu, my_tok, r);
      head = __shfl_sync(0xffffffffu, my_head, r);
      return tok < s.n;
    };

    // Q as the second operand: tile t's row 8 t + i8, of which lane j has D / 4 neighbouring channels, 8 of
    // them in two products. With four tiles it would take a quarter of the registers: warp t prepares
    // tile t, and all read it from shared memory.
    constexpr bool kSharedQ = NT == 4;
    constexpr int kOwnQ = kSharedQ ? 1 : NT;
    uint32_t q[kOwnQ][D / 16][2];
#pragma unroll
    for (int t = 0; t < kOwnQ; ++t) {
      int tok, head;
      const bool on = row(8 * (kSharedQ ? warp : t) + i8, tok, head);
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + (static_cast<long long>(p.h * a.group + (on ? head : 0)) * a.c.total_new + s.a + (on ? tok : 0)) * D);
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        const uint4 v = on ? load(src + (D / 32) * j + w) : make_uint4(0, 0, 0, 0);
        q[t][2 * w][0] = v.x;
        q[t][2 * w][1] = v.y;
        q[t][2 * w + 1][0] = v.z;
        q[t][2 * w + 1][1] = v.w;
      }
    }

    // This lane's 16 bytes of the head's rows (row lane / kPieces and every 32 / kPieces-th after it) and of
    // its scales, in page 0. Scales are an eighth of the codes, wherever they lie.
    const long long page_bytes = (static_cast<long long>(a.c.hkv) * C::kRowBytes) << a.c.page_shift;
    const long long in_head = (static_cast<long long>(p.h) * C::kRowBytes) << a.c.page_shift;
    const uint8_t* lane_k = a.c.k_pages + in_head + 16 * lane;
    const uint8_t* lane_v = a.c.v_pages + in_head + 16 * lane;
    const uint8_t* lane_s = (scales_of_v ? a.c.v_scales : a.c.k_scales) + in_head / 8 + scale_at;
    int n_issued = 0, issue_stage = 0;
    auto issue = [&]() {
      const int key = key0 + n_issued * (kKeys * kWarps);
      if (key < kend) {
        if ((n_issued & 15) == 0 && n_issued > 0) {
          pages = pages_next;
          pages_next = entries(p, (n_issued >> 4) + 1);
        }
        constexpr int kPer = 32 / C::kPieces, kX = kChunk / kPer;  // rows of one instruction, instructions of a chunk
        const uint32_t dst = stages + issue_stage * C::kStage, scales = dst + 2 * C::kTile + 16 * lane;
        const int r = lane / C::kPieces, c = lane % C::kPieces;
        long long at[2];
        bool ok[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int page = __shfl_sync(0xffffffffu, pages, 2 * (n_issued & 15) + u);
          ok[u] = static_cast<unsigned>(page) < static_cast<unsigned>(a.c.n_pages);
          at[u] = static_cast<unsigned>(page) * page_bytes + ((key + kChunk * u) & page_mask) * C::kRowBytes;
        }
        const uint8_t* from = lane_s + (scale_chunk ? at[1] : at[0]) / 8;
        if (ok[0] && ok[1] && key + kKeys <= s.len) {
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int x = 0; x < kX; ++x) {
              const int to = piece_at<C::kRowBytes>((u * kX + x) * kPer + r, c);
              cp_async16(dst + to, lane_k + at[u] + x * kPer * C::kRowBytes);
              cp_async16(dst + C::kTile + to, lane_v + at[u] + x * kPer * C::kRowBytes);
            }
          if (lane < 2 * kScalePieces) cp_async16(scales, from);
        } else {  // rows behind the last key may hold anything: zeros come in their place, and in their scales'
#pragma unroll 1
          for (int u = 0; u < 2; ++u) {
            const bool there = u ? ok[1] : ok[0];
            const int first = key + kChunk * u;
            if (!there && first < s.len && lane == 0) atomicCAS(a.c.status, 0, kErrCachePage);
#pragma unroll 1
            for (int x = 0; x < kX; ++x) {
              const bool on = there && first + x * kPer + r < s.len;
              const int to = piece_at<C::kRowBytes>((u * kX + x) * kPer + r, c);
              const long long off = (u ? at[1] : at[0]) + x * kPer * C::kRowBytes;
              cp_async16_or_zeros(dst + to, on ? lane_k + off : a.c.k_pages, on);
              cp_async16_or_zeros(dst + C::kTile + to, on ? lane_v + off : a.c.v_pages, on);
            }
          }
          const int held = (s.len - key - kChunk * scale_chunk) * C::kScales - scale_at;
          const int bytes = (scale_chunk ? ok[1] : ok[0]) ? min(max(held, 0), 16) : 0;
          if (lane < 2 * kScalePieces) cp_async16_part(scales, bytes > 0 ? from : a.c.k_scales, bytes);
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

    // Q's rows as f16 scaled by 2^(14 - e), e the largest exponent of the row (exact but for elements 2^-28
    // times the largest); `back` takes the scores of row i8 of a tile to log2 units.
    float back[kOwnQ];
#pragma unroll
    for (int t = 0; t < kOwnQ; ++t) {
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
      // Neither zero, which would make NaN of a masked score (what this does to others is below 2^-80), nor
      // infinite, which would of a score of zero (others may be wrong then: they are past what the header allows).
      back[t] = fminf(fmaxf(a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - up) << 23), 0x1p-120f), 0x1p127f);
    }
    if constexpr (kSharedQ) {
#pragma unroll
      for (int c = 0; c < D / 16; ++c) shared_q[warp][c][lane] = make_uint2(q[0][c][0], q[0][c][1]);
      if (j == 0) shared_back[8 * warp + i8] = back[0];
      __syncthreads();
    }
    auto q_of = [&](int t, int c) -> uint2 {
      if constexpr (kSharedQ) return shared_q[t][c][lane];
      else return make_uint2(q[t][c][0], q[t][c][1]);
    };
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
        else factor[t][e] = __shfl_sync(0xffffffffu, back[t], 4 * (2 * j + e));
      }

    // m: the maximum of a row's scores less kUp, which its weights are relative to (`less` is -m, or 0 for a
    // row without a key yet); the eight lanes of a column pair share it. l: the weights' sum over the
    // lane's own keys.
    float m[NT][2], less[NT][2], l[NT][2], acc[D / 16][NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[t][e] = -INFINITY;
        less[t][e] = l[t][e] = 0.f;
      }
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[c][t][e] = 0.f;
    }

    int stage = 0;
    for (int key = key0; key < kend; key += kKeys * kWarps) {
      cp_wait<C::kStages - 2>();
      __syncwarp();  // this stage has arrived, and every lane is done with the one that is filled next
      issue();
      const uint32_t kt = stages + stage * C::kStage, vt = kt + C::kTile;
      const uint32_t ks = vt + C::kTile, vs = ks + C::kScaleTile;
      stage = stage + 1 == C::kStages ? 0 : stage + 1;
      float sc[2][NT][4];  // S^T: element 2 y + e is key `key` + 16 u + 8 y + i8, row 8 t + 2 j + e
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[u][t][e] = 0.f;
        const int r = kChunk * u + i8;
        uint32_t raw[2][D / 32], scale[2];  // of keys r and r + 8: 8 codes to a word; scales of the words' halves
        if constexpr (D == 128) {
          const uint4 v0 = lds16(kt + piece_at<C::kRowBytes>(r, j)), v1 = lds16(kt + piece_at<C::kRowBytes>(r + 8, j));
          raw[0][0] = v0.x, raw[0][1] = v0.y, raw[0][2] = v0.z, raw[0][3] = v0.w;
          raw[1][0] = v1.x, raw[1][1] = v1.y, raw[1][2] = v1.z, raw[1][3] = v1.w;
          const uint32_t s0 = lds_u16(ks + r * 8 + 2 * j), s1 = lds_u16(ks + (r + 8) * 8 + 2 * j);
          e4m3x4_to_f16x2(__byte_perm(s0, s1, 0x5410), scale[0], scale[1]);
        } else {
          const uint2 v0 = lds8(kt + piece_at<C::kRowBytes>(r, j >> 1) + 8 * (j & 1));
          const uint2 v1 = lds8(kt + piece_at<C::kRowBytes>(r + 8, j >> 1) + 8 * (j & 1));
          raw[0][0] = v0.x, raw[0][1] = v0.y;
          raw[1][0] = v1.x, raw[1][1] = v1.y;
          const uint32_t s0 = lds_u8(ks + r * 4 + j), s1 = lds_u8(ks + (r + 8) * 4 + j);
          e4m3x4_to_f16x2(__byte_perm(s0, s1, 0x4400), scale[0], scale[1]);
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          uint32_t f0[4], f1[4];
          e2m1x8_to_f16x2(raw[0][w], f0);
          e2m1x8_to_f16x2(raw[1][w], f1);
          const uint32_t x0 = half_of(scale[0], w >> 1), x1 = half_of(scale[1], w >> 1);
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const uint32_t f[4] = {mul_f16x2(f0[2 * z], x0), mul_f16x2(f1[2 * z], x1), mul_f16x2(f0[2 * z + 1], x0),
                                   mul_f16x2(f1[2 * z + 1], x1)};
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const uint2 y = q_of(t, 2 * w + z);
              mma16816h(sc[u][t], f, y.x, y.y);
            }
          }
        }
      }
      if (key + kKeys > lim_min) {  // some row does not see all of this
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (key + kChunk * u + 8 * (e >> 1) + i8 >= lim[t][e & 1]) sc[u][t][e] = -INFINITY;
        // A NaN scale of V must not meet the zero weights of rows that do not see it: zeros take its place,
        // and the channels of the rows that do see it become NaN here.
        constexpr int kCount = kKeys * C::kScales;
        bool nan = false;
        for (int x = 4 * lane; x < kCount; x += 128) {
          const uint32_t four = lds4(vs + x);
          nan = nan || (((four & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0u;
        }
        if (__any_sync(0xffffffffu, nan)) {
#pragma unroll 1
          for (int x = 0; x < kCount; ++x) {  // key x / kScales, group x % kScales
            if ((lds_u8(vs + x) & 0x7fu) != 0x7fu) continue;
            __syncwarp();
            if (lane == 0) asm volatile("st.shared.u8 [%0], %1;" ::"r"(vs + x), "r"(0) : "memory");
            const int g = x % C::kScales;
#pragma unroll
            for (int c = 0; c < D / 16; ++c)
              if (g == 2 * (c >> 1) + (lane >> 4))
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    if (key + x / C::kScales < lim[t][e & 1]) acc[c][t][e] = __uint_as_float(0x7fc00000u);
          }
          __syncwarp();
        }
      }
      // raise the running maxima only when some row's grew by more than 2^8
      bool grow = false;
      float top[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[t][e] = max3f(fmaxf(sc[0][t][e], sc[0][t][2 + e]), sc[1][t][e], sc[1][t][2 + e]);
          top[t][e] *= factor[t][e];
          grow = grow || top[t][e] > m[t][e] + (kGrow + kUp);
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float to = top[t][e] - kUp;
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, o));
            to = fmaxf(to, m[t][e]);
            const float f = to == -INFINITY ? 1.f : fast_exp2(m[t][e] - to);
            m[t][e] = to;
            less[t][e] = to == -INFINITY ? 0.f : -to;
            l[t][e] *= f;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              acc[c][t][e] *= f;
              acc[c][t][2 + e] *= f;
            }
          }
      }
      // P^T: the packed pairs are (key; rows 2 j, 2 j + 1) and are wanted as (row; keys 2 j, 2 j + 1). In f16:
      // off by 2^-11 of itself, or 2^-25 where the row's largest weight is 2^7 at least.
      uint32_t pt[2][NT][2];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float2 x = ffma2(sc[u][t][2 * y], sc[u][t][2 * y + 1], factor[t][0], factor[t][1], less[t][0], less[t][1]);
            const float p0 = fast_exp2(x.x), p1 = fast_exp2(x.y);
            const float2 sum = fadd2(l[t][0], l[t][1], p0, p1);
            l[t][0] = sum.x;
            l[t][1] = sum.y;
            pt[u][t][y] = transpose8x8(pack_f16(p0, p1));
          }
#pragma unroll
      for (int u = 0; u < 2; ++u)
        each_v<D>(vt + kChunk * u * C::kRowBytes, vs + kChunk * u * C::kScales, lane,
                  [&](int c, const uint32_t(&v)[4]) {
#pragma unroll
                    for (int t = 0; t < NT; ++t) mma16816h(acc[c][t], v, pt[u][t][0], pt[u][t][1]);
                  });
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
        f *= a.c.v_unit;
        float* dst = sums + (static_cast<size_t>(warp) * kRows + r) * kSumRow;
#pragma unroll
        for (int c = 0; c < D / 16; ++c)  // channels as each_v has them
          *reinterpret_cast<float2*>(dst + 32 * (c >> 1) + 4 * i8 + 2 * (c & 1)) =
              make_float2(acc[c][t][e] * f, acc[c][t][2 + e] * f);
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

template <int D, int NT>
fcp_status launch(AttnArgs a, void* workspace, int dev, int n_sm, int max_new, cudaStream_t s) {
  using C = Cfg<D, NT>;
  using P = Rows<NT>;
  constexpr int kSmem = std::max(kWarps * C::kWarpBytes, kWarps * P::kRows * (D + 4) * 4);
  const int blocks = std::min(kPerSm<NT> * n_sm, kMaxBlocks);
  set_workspace<P>(a, workspace, D, kMaxBlocks);
  static std::atomic<uint64_t> allowed{0};
  if (const fcp_status st = allow_smem(few4_kernel<D, NT>, kSmem, dev, allowed, "paged attention smem attribute");
      st != FCP_OK)
    return st;
  if (const fcp_status st = launch_overlapped(few4_kernel<D, NT>, dim3(blocks), kFewThreads, kSmem, s,
                                              "paged attention launch", a);
      st != FCP_OK)
    return st;
  // the merge's row slices, as in fcp_paged_few.cu
  const long long rows = std::min<long long>(static_cast<long long>(std::max(max_new, 1)) * a.group, P::kRows);
  const bool few_pieces = static_cast<long long>(P::kWarpPieces) * a.c.n_seqs * a.c.hkv >= blocks;
  return launch_merge<P, D>(
      a, blocks, static_cast<int>(few_pieces ? (rows + 2 * kMergeWarps - 1) / (2 * kMergeWarps) : rows), s);
}

template <int D>
fcp_status launch_rows(const AttnArgs& a, int rows, void* workspace, int dev, int n_sm, int max_new, cudaStream_t s) {
  return rows <= 8    ? launch<D, 1>(a, workspace, dev, n_sm, max_new, s)
         : rows <= 16 ? launch<D, 2>(a, workspace, dev, n_sm, max_new, s)
                      : launch<D, 4>(a, workspace, dev, n_sm, max_new, s);
}

}  // namespace

fcp_status launch_paged_few4(const AttnArgs& a, int d, int rows, void* workspace, int dev, int n_sm, int max_new,
                             cudaStream_t s) {
  return d == 128 ? launch_rows<128>(a, rows, workspace, dev, n_sm, max_new, s)
                  : launch_rows<64>(a, rows, workspace, dev, n_sm, max_new, s);
}

}  // namespace fcp
