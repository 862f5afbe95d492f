// Rotary positions: pairs of channels turned by position * frequency, of q and k as they are, or of a
// batch's new tokens with the turned k and v going straight to a paged cache.
//
// (a, b) -> m (a cos x - b sin x, b cos x + a sin x) with x = position * f. The frequencies come as turns
// a position in units of 2^-64, so position * f modulo a whole turn is the low half of one integer
// product, right to 2^-32 of a turn at any position, where a float32 product is off by tenths of
// a radian at positions past 10^6. cos and sin are worked out once for a token and serve all the
// heads that a block does: a thread keeps those of its 8 pairs (16 channels of a row) and goes from
// head to head, four rows in flight.
//
// Bound by HBM: every row is read and written once. Measured: 32768 tokens of 64 + 8 heads, D = 128, 180 us
// (6710 GB/s, a copy's rate; both pairings, and half of the head turned, the same; D = 64 92 us, 98%);
// 14000 tokens placed in a bf16 cache 103.6 us (6260 GB/s, 93%), in an e4m3 one 106 (86%), in 4 bits 117 (77%;
// the quantisation's instructions; 137 with two blocks to an SM instead of three and the neighbours that share
// a scale worked out for each row). Four blocks to an SM 184, 107, 108 and 122 us. Small calls are the
// host's 8 us; as part of a graph 4 to 6.
#include <algorithm>
#include <cmath>

#include "fcp_move.cuh"

namespace fcp {
namespace {

constexpr int kRows = 4;    // rows that a thread has in flight
constexpr int kNone = -1;   // no cache
constexpr int kBlocks = 8;  // blocks to an SM that the heads are split for

struct RotaryArgs {
  PagedArgs c;
  const int32_t* positions;
  const uint64_t* turns;
  float magnitude;
  int32_t part, interleaved, back;
  const uint4 *q, *k, *v;
  uint4 *q_out, *k_out;
  int32_t hq, hkv, heads, total;  // heads: of q, k and v that a block does
};

// 8 channels as float32, and back.
__device__ __forceinline__ void unpack(const uint4 x, float (&y)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[2 * i] = __uint_as_float(w[i] << 16);
    y[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack(const float (&y)[8]) {
  return make_uint4(dev::pack_bf16(y[0], y[1]), dev::pack_bf16(y[2], y[3]), dev::pack_bf16(y[4], y[5]),
                    dev::pack_bf16(y[6], y[7]));
}

// m cos and m sin of phase / 2^32 turns, off by 0.26 units in the last place on average (rounding alone: 0.25)
// and 1.6 at most: the nearest quarter turn is taken off, what is left, x within an eighth of a turn, is kept as a sum of
// two numbers, and the series of sin x - x and cos x - 1 (Taylor's, whose first terms left out are below
// 2^-29) are added to what is exact, in one rounding with the product by m. (sincospif
// of the phase as float32 changed the rounding to bf16 of more of the k that a cache keeps.)
__device__ __forceinline__ void turn_by(uint32_t phase, float m, float& c, float& s) {
  const uint32_t quarter = (phase + (1u << 29)) >> 30;
  const int rest = static_cast<int>(phase - (quarter << 30));  // -2^29 .. 2^29 - 1
  const float high = static_cast<float>(rest);
  const float low = static_cast<float>(rest - static_cast<int>(high));
  // 2 pi 2^-32 as a sum of two float32
  constexpr double kTurn = 6.283185307179586476925 / 4294967296.0;
  constexpr float k0 = static_cast<float>(kTurn), k1 = static_cast<float>(kTurn - static_cast<double>(k0));
  const float x = high * k0;
  const float dx = fmaf(high, k0, -x) + fmaf(high, k1, low * k0);
  const float y = x * x;
  const float sx = fmaf(fmaf(fmaf(2.7557319e-6f, y, -1.9841270e-4f), y, 8.3333333e-3f), y, -1.6666667e-1f) * y;  // sin x / x - 1
  const float cx = fmaf(fmaf(fmaf(fmaf(-2.7557319e-7f, y, 2.4801587e-5f), y, -1.3888889e-3f), y, 4.1666667e-2f), y, -0.5f) * y;
  // cos x has an error of y's rounding, y = x^2 - dy, that is halved
  const float dy = fmaf(x, x, -y);
  const float sin_m = fmaf(m, x, m * fmaf(x, sx, dx));
  const float cos_m = fmaf(m, 1.f, m * (cx - fmaf(0.5f, dy, x * dx)));
  const float a = quarter & 1u ? sin_m : cos_m, b = quarter & 1u ? cos_m : sin_m;
  c = (quarter + 1u) & 2u ? -a : a;
  s = quarter & 2u ? -b : b;
}

// grid (ceil(T / 32), slices of the heads)
template <int D, int kKind>
__global__ void __launch_bounds__(kMoveThreads, 3) rotary_kernel(const RotaryArgs a) {
  constexpr int kLanes = D / 16, kRow = D / 8;                   // threads of a row; 16-byte chunks of it
  constexpr int kGroups = kMoveThreads / (kLanes * kMoveTokens);  // rows of a token at a time
  constexpr bool kCache = kKind != kNone;
  __shared__ TokenPlace place[kMoveTokens];
  __shared__ int coarse[kCache ? kCoarse : 1], lens[kCache ? kCoarse : 1];
  let_next_start();
  wait_for_previous();
  const int l = threadIdx.x % kLanes, tok = threadIdx.x / kLanes % kMoveTokens, group = threadIdx.x / (kLanes * kMoveTokens);
  const int t0 = blockIdx.x * kMoveTokens, t = t0 + tok;
  int pos = 0, page = -1, off = 0;
  bool on = t < a.total;
  if constexpr (kCache) {
    find_places(a.c, t0, place, coarse, lens);
    if (blockIdx.x + blockIdx.y == 0)  // errors of sequences that no row is found in, too
      for (int i = threadIdx.x; i < a.c.n_seqs; i += kMoveThreads) seq_shape(a.c, i, true);
    pos = place[tok].pos;
    page = place[tok].page;
    off = place[tok].off;
    on = on && pos >= 0;
  } else if (on) {
    pos = load(a.positions + t);
  }

  // This thread's two chunks of a row, A and B, and its 8 pairs: channel 8 A + i with 8 B + i, or
  // neighbours, four in each. Chunks behind the turned part go as they are.
  int at[2];
  bool turned[2];
  const int lanes = a.part >> 4;  // threads that turn, where a pair's channels are part / 2 apart
  if (a.interleaved) {
    at[0] = l;
    at[1] = kLanes + l;
    turned[0] = 8 * at[0] < a.part;
    turned[1] = 8 * at[1] < a.part;
  } else {
    turned[0] = turned[1] = l < lanes;
    at[0] = l < lanes ? l : 2 * lanes + (l - lanes);
    at[1] = l < lanes ? lanes + l : 2 * lanes + (kLanes - lanes) + (l - lanes);
  }
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int pair = a.interleaved ? 4 * at[i >> 2] + (i & 3) : 8 * l + i;
    c[i] = 1.f;
    s[i] = 0.f;
    if (on && turned[i >> 2]) {
      const uint64_t x = static_cast<uint64_t>(static_cast<int64_t>(pos)) * a.turns[pair];
      turn_by(static_cast<uint32_t>(x >> 32), a.magnitude, c[i], s[i]);
      if (a.back) s[i] = -s[i];
    }
  }
  auto turn = [&](uint4 (&x)[2]) {
    float y[2][8], z[2][8];
    unpack(x[0], y[0]);
    unpack(x[1], y[1]);
    if (a.interleaved) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float u = y[h][2 * i], w = y[h][2 * i + 1];
          z[h][2 * i] = fmaf(u, c[4 * h + i], -(w * s[4 * h + i]));
          z[h][2 * i + 1] = fmaf(w, c[4 * h + i], u * s[4 * h + i]);
        }
        if (turned[h]) x[h] = pack(z[h]);
      }
    } else if (turned[0]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        z[0][i] = fmaf(y[0][i], c[i], -(y[1][i] * s[i]));
        z[1][i] = fmaf(y[1][i], c[i], y[0][i] * s[i]);
      }
      x[0] = pack(z[0]);
      x[1] = pack(z[1]);
    }
  };
  // e2m1: the 8 channels that share a scale with a chunk's are the chunk at ^ 1: the lane that has it, as which
  // of its two.
  int from[2] = {}, which[2] = {};
  if constexpr (kKind == FCP_CACHE_E2M1) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int other = at[h] ^ 1, rest = kLanes - lanes;
      if (a.interleaved) {
        which[h] = other >= kLanes;
        from[h] = which[h] ? other - kLanes : other;
      } else if (other < 2 * lanes) {
        which[h] = other >= lanes;
        from[h] = which[h] ? other - lanes : other;
      } else {
        which[h] = other - 2 * lanes >= rest;
        from[h] = lanes + (other - 2 * lanes) - (which[h] ? rest : 0);
      }
      from[h] += (threadIdx.x & 31) - l;
    }
  }
  // Two chunks of a row of the cache.
  auto store = [&](const uint4 (&x)[2], int head, bool is_v) {
    if constexpr (kCache) {
      const long long row = (page >= 0 ? page_row(a.c, page, head) : 0) + off;
      uint8_t* pages = is_v ? a.c.v_pages : a.c.k_pages;
      uint8_t* scales = is_v ? a.c.v_scales : a.c.k_scales;
      const bool there = on && page >= 0;
      if constexpr (kKind == FCP_CACHE_BF16) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (there) reinterpret_cast<uint4*>(pages)[row * kRow + at[h]] = x[h];
      } else if constexpr (kKind == FCP_CACHE_E4M3) {
        uint32_t two = max_u16x2(top_pair(x[0]), top_pair(x[1]));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) two = max_u16x2(two, __shfl_xor_sync(0xffffffffu, two, o));
        uint32_t byte = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint2 codes = quantise8(x[h], max(two & 0xffffu, two >> 16), byte);
          if (there) reinterpret_cast<uint2*>(pages)[row * kRow + at[h]] = codes;
        }
        if (there && l == 0) scales[row] = static_cast<uint8_t>(byte);
      } else {
        const float per_unit = 1.f / (is_v ? a.c.v_unit : a.c.k_unit);
        const uint32_t top[2] = {top_pair(x[0]), top_pair(x[1])};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t u = __shfl_sync(0xffffffffu, top[0], from[h]), w = __shfl_sync(0xffffffffu, top[1], from[h]);
          const uint32_t two = max_u16x2(top[h], which[h] ? w : u);
          uint32_t byte;
          const uint32_t codes = quantise4(x[h], max(two & 0xffffu, two >> 16), per_unit, byte);
          if (there) {
            reinterpret_cast<uint32_t*>(pages)[row * kRow + at[h]] = codes;
            if ((at[h] & 1) == 0) scales[row * (D / 16) + at[h] / 2] = static_cast<uint8_t>(byte);
          }
        }
      }
    }
  };

  const int all = a.hq + a.hkv * (kCache ? 2 : 1);
  const int h1 = min(static_cast<int>(blockIdx.y + 1) * a.heads, all);
  const long long step = static_cast<long long>(a.total) * kRow, mine = static_cast<long long>(t) * kRow;
  for (int h0 = blockIdx.y * a.heads + group; h0 < h1; h0 += kRows * kGroups) {
    uint4 x[kRows][2];
#pragma unroll
    for (int y = 0; y < kRows; ++y) {
      const int h = h0 + y * kGroups;
      x[y][0] = x[y][1] = make_uint4(0u, 0u, 0u, 0u);
      if (!on || h >= h1) continue;
      const uint4* src = h < a.hq           ? a.q + h * step
                         : h < a.hq + a.hkv ? a.k + (h - a.hq) * step
                                            : a.v + (h - a.hq - a.hkv) * step;
      x[y][0] = __ldcs(src + mine + at[0]);
      x[y][1] = __ldcs(src + mine + at[1]);
    }
#pragma unroll
    for (int y = 0; y < kRows; ++y) {
      const int h = h0 + y * kGroups;
      if (h >= h1) break;  // the same for a whole warp
      if (h < a.hq + a.hkv) turn(x[y]);
      if (h < a.hq || !kCache) {
        uint4* dst = h < a.hq ? a.q_out + h * step : a.k_out + (h - a.hq) * step;
        if (on) {
          __stcs(dst + mine + at[0], x[y][0]);
          __stcs(dst + mine + at[1], x[y][1]);
        }
      } else {
        store(x[y], h < a.hq + a.hkv ? h - a.hq : h - a.hq - a.hkv, h >= a.hq + a.hkv);
      }
    }
  }
}

fcp_status rotary_args(const fcp_rotary* r, int head_dim, RotaryArgs* a) {
  if (r == nullptr || !r->turns || (reinterpret_cast<uintptr_t>(r->turns) & 7u) != 0) return FCP_ERR_INVALID;
  if (r->rotary_dim <= 0 || r->rotary_dim > head_dim || !(r->magnitude > 0.f) || !std::isfinite(r->magnitude))
    return FCP_ERR_INVALID;
  if (r->rotary_dim % 16 != 0) return FCP_ERR_UNSUPPORTED;
  a->turns = r->turns;
  a->magnitude = r->magnitude;
  a->part = r->rotary_dim;
  a->interleaved = r->interleaved ? 1 : 0;
  return FCP_OK;
}

// The heads are split over blocks until those fill the GPU some times over; a launch that overlaps the
// kernel before it costs the host another microsecond and a half, which is worth it from there on.
template <int D, int kKind>
fcp_status launch(RotaryArgs& a, cudaStream_t s) {
  int dev = 0, n_sm = 0;
  if (const fcp_status st = this_device(&dev, &n_sm); st != FCP_OK) return st;
  const int all = a.hq + a.hkv * (kKind != kNone ? 2 : 1);
  const unsigned bx = static_cast<unsigned>((a.total + kMoveTokens - 1) / kMoveTokens);
  constexpr int kGroups = 128 / D;
  auto slices = [&](int heads) { return (all + heads - 1) / heads; };
  a.heads = all;
  while (a.heads > kGroups && static_cast<long long>(bx) * slices(a.heads) < kBlocks * n_sm) a.heads = (a.heads + 1) / 2;
  const dim3 grid(bx, static_cast<unsigned>(slices(a.heads)));
  if (static_cast<long long>(bx) * slices(a.heads) >= kBlocks * n_sm)
    return launch_overlapped(rotary_kernel<D, kKind>, grid, kMoveThreads, 0, s, "rotary launch", a);
  rotary_kernel<D, kKind><<<grid, kMoveThreads, 0, s>>>(a);
  FCP_CUDA_TRY(cudaGetLastError(), "rotary launch");
  return FCP_OK;
}

}  // namespace
}  // namespace fcp

using namespace fcp;

extern "C" fcp_status fcp_rotary_apply(const fcp_rotary* rotary, const int32_t* positions, int32_t total, const void* q,
                                       void* q_out, int32_t hq, const void* k, void* k_out, int32_t hkv,
                                       int32_t head_dim, int32_t backward, void* stream) {
  RotaryArgs a = {};
  if (total < 0 || hq < 0 || hkv < 0) return FCP_ERR_INVALID;
  if (head_dim != 64 && head_dim != 128) return FCP_ERR_UNSUPPORTED;
  if (const fcp_status st = rotary_args(rotary, head_dim, &a); st != FCP_OK) return st;
  if (total > 1 << 30 || hq > 65535 || hkv > 65535) return FCP_ERR_UNSUPPORTED;
  if (total == 0 || hq + hkv == 0) return FCP_OK;
  if (!positions || !aligned4(positions)) return FCP_ERR_INVALID;
  if (hq > 0 && (!q || !q_out || !aligned16(q) || !aligned16(q_out))) return FCP_ERR_INVALID;
  if (hkv > 0 && (!k || !k_out || !aligned16(k) || !aligned16(k_out))) return FCP_ERR_INVALID;
  a.positions = positions;
  a.back = backward ? 1 : 0;
  a.q = static_cast<const uint4*>(q);
  a.k = static_cast<const uint4*>(k);
  a.q_out = static_cast<uint4*>(q_out);
  a.k_out = static_cast<uint4*>(k_out);
  a.hq = hq;
  a.hkv = hkv;
  a.total = total;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return head_dim == 128 ? launch<128, kNone>(a, s) : launch<64, kNone>(a, s);
}

extern "C" fcp_status fcp_rotary_write(const fcp_cache* cache, const fcp_cache_batch* batch, const fcp_rotary* rotary,
                                       const void* q, void* q_out, int32_t hq, const void* k, const void* v,
                                       void* stream) {
  RotaryArgs a = {};
  if (const fcp_status st = paged_args(cache, batch, &a.c); st != FCP_OK) return st;
  if (hq < 0) return FCP_ERR_INVALID;
  if (const fcp_status st = rotary_args(rotary, cache->head_dim, &a); st != FCP_OK) return st;
  if (hq > 65535 || cache->hkv > 65535) return FCP_ERR_UNSUPPORTED;
  if (a.c.total_new == 0 || a.c.n_seqs == 0) return FCP_OK;
  if (hq > 0 && (!q || !q_out || !aligned16(q) || !aligned16(q_out))) return FCP_ERR_INVALID;
  if (!k || !v || !aligned16(k) || !aligned16(v)) return FCP_ERR_INVALID;
  a.q = static_cast<const uint4*>(q);
  a.k = static_cast<const uint4*>(k);
  a.v = static_cast<const uint4*>(v);
  a.q_out = static_cast<uint4*>(q_out);
  a.hq = hq;
  a.hkv = cache->hkv;
  a.total = a.c.total_new;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool wide = cache->head_dim == 128;
  if (cache->dtype == FCP_CACHE_E2M1) return wide ? launch<128, FCP_CACHE_E2M1>(a, s) : launch<64, FCP_CACHE_E2M1>(a, s);
  if (cache->dtype == FCP_CACHE_E4M3) return wide ? launch<128, FCP_CACHE_E4M3>(a, s) : launch<64, FCP_CACHE_E4M3>(a, s);
  return wide ? launch<128, FCP_CACHE_BF16>(a, s) : launch<64, FCP_CACHE_BF16>(a, s);
}
