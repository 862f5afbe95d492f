// Attention of chunks of new tokens over a paged cache on sm_103a (tcgen05 + TMEM).
//
// A unit is up to two tiles of 128 rows of one KV head, each of 16, 32, 64 or 128 new tokens of as
// many query heads of the group as fill it, and every key tile loaded serves all of a unit's
// rows. Rows are computed independently of one another: those past the chunk or the group hold
// whatever is in shared memory and are not stored.
//
// As in the forward over a work list, S_t = Q_t K^T and O_t += P_t V run on the tensor core
// with accumulators in tensor memory while the other tile's softmax runs; what differs is where
// keys come from. A key tile is 128 positions, gathered from their pages into the
// 128-byte-swizzled layout that the matrix instructions read: a bf16 cache by TMA, one box for
// each page and 64 channels, an e4m3 cache by six warps that turn codes into scaled bf16 on
// their way to shared memory. That product with a power of two is exact, so the kernel computes
// the attention over what reading the cache gives, and the tensor core runs the same bf16
// instructions for both. Rows of V past the sequence become zeros, since a zero weight times
// whatever such a row holds may be NaN. So do an e4m3 cache's NaN rows of V, which rows that come
// before them must not meet: a unit keeps the first position of one, and o of the rows that see it
// becomes NaN when it is stored.
//
// Bound by the chain of each key tile, S -> softmax -> P -> PV, as the forward is: tensor memory has
// no room for a second S of a tile; an e4m3 cache adds the loaders' instructions to the softmax's.
// Measured (64 query, 8 KV heads, D = 128, alone): 2048 new tokens over 32768 keys 1330 us from a bf16
// cache (1600 TFLOP/s) and 1710 us from an e4m3 one (1245), 8192 over 8192 735 and 965 us, 16 chunks
// of 512 with nothing before them 156 and 192 us (a quarter of it writes o; what a unit costs beside
// its one to four key tiles is most of the rest). Call after call the first two are 1440 to 1520 and
// 1880 us: blocks then land on other SMs, and the slowest decides.
//
// Warps 0-3 and 4-7: softmax of tile 0 and 1 (thread = row = TMEM lane); 8: the walk along the
// block's share of the work, Q's loads and a bf16 cache's; 9: MMA; 10-15 (e4m3 only): loaders.
// TMEM columns: S_t at [128 t, 128 t + 128), overwritten by P_t as bf16; O_t at [256 + 128 t,
// 256 + 128 t + D).
#include <algorithm>
#include <cmath>

#include "fcp_paged_sched.cuh"

namespace fcp {
namespace {

using namespace dev;

constexpr int kLoaders = 6;  // warps
template <bool kE4M3>
constexpr int kThreads = 32 * (10 + (kE4M3 ? kLoaders : 0));
constexpr int kPanelBytes = kTileM * 128;  // 128 rows x 64 bf16 channels
constexpr float kRescaleThreshold = 8.0f;   // log2 units
constexpr int kQBox = 16;                   // tokens of a TMA load of Q for tiles of several heads
// Registers a thread with the loader warps: the launch gives 128, and the softmax warps take
// what the others leave (they hold a row of 128 scores).
constexpr int kRegsSoftmax = 168, kRegsOther = 88;
static_assert(2 * kRegsSoftmax + 2 * kRegsOther <= 4 * 128, "the split fits the launch's registers");

enum : int {
  B_QFULL = 0,
  B_QEMPTY = 1,  // the S MMAs of a unit have read Q
  B_KFULL = 2,   // 2 stages
  B_KEMPTY = 4,
  B_VFULL = 6,
  B_VEMPTY = 8,
  B_SFULL = 10,  // per tile
  B_PFULL = 12,  // per tile and half: keys [0, 64) and [64, 128) of P are in TMEM
  B_ODONE = 16,  // per tile
  B_OFREE = 18,  // per tile: the epilogue has read O_t out of TMEM
  B_DRAIN = 20,
  B_TFULL = 21,   // 2 slots: the next unit is published
  B_TEMPTY = 23,  // 2 slots: the MMA, softmax and loader warps have read it
  B_COUNT = 25
};

// A block's piece of a group: key tiles [kt0, kt1) of unit u.
struct Unit {
  int valid, i, a, n, len, h, u, kt0, kt1, slot, pad0, pad1;
};
constexpr int kNanKeyOff = B_COUNT * 8 + 12;  // of the last 4 units: the first key whose row of V is NaN
constexpr int kUnitOff = 256;
constexpr int kBarArea = kUnitOff + 2 * static_cast<int>(sizeof(Unit));
static_assert(kNanKeyOff + 4 * 4 <= kUnitOff, "barrier area");

template <int D>
struct Cfg {
  static constexpr int kTileBytes = kTileM * D * 2;
  static constexpr int kPanels = D / 64;
  static constexpr int kQ = 0;                     // 2 tiles
  static constexpr int kK = 2 * kTileBytes;        // 2 stages
  static constexpr int kV = 4 * kTileBytes;        // 2 stages
  static constexpr int kBar = 6 * kTileBytes;
  static constexpr int kStage = kBar + kBarArea;   // epilogue: 32 rows x 128 bytes per softmax warp
  static constexpr int kStageBytes = 8 * 32 * 128;
  static constexpr int kEnd = kStage + kStageBytes;
  // at least half the SM's shared memory, so one block per SM holds all 512 TMEM columns
  static constexpr int kSmemBytes = kEnd > 118 * 1024 ? kEnd : 118 * 1024;
  static_assert(kStage % 16 == 0, "16-byte aligned staging");
  static_assert(kSmemBytes <= 232448, "shared memory per block");
  static constexpr uint32_t kIdescS = idesc_bf16(kTileM, kTileN, false, false);
  static constexpr uint32_t kIdescPV = idesc_bf16(kTileM, D, false, true);
};

// 8 codes times 2^-120 as bf16: a code's exponent and mantissa moved to bf16's fields, four codes
// at a time (the high bytes, the low bytes, then interleaved).
__device__ __forceinline__ void code_bits(const uint2 x, uint32_t (&r)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w = i ? x.y : x.x;
    const uint32_t hi = (w & 0x80808080u) | ((w >> 4) & 0x07070707u), lo = (w & 0x0f0f0f0fu) * 16u;
    r[2 * i] = __byte_perm(lo, hi, 0x5140);
    r[2 * i + 1] = __byte_perm(lo, hi, 0x7362);
  }
}
__device__ __forceinline__ void times(uint32_t (&r)[4], uint32_t f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 y =
        __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&r[i]), *reinterpret_cast<const __nv_bfloat162*>(&f));
    r[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
}

template <int D, bool kE4M3>
__global__ void __launch_bounds__(kThreads<kE4M3>, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmQ16,
                 const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV, const AttnArgs a) {
  constexpr int kThreads = fcp::kThreads<kE4M3>;
  using C = Cfg<D>;
  using P = ChunkRows;
  extern __shared__ __align__(1024) uint8_t smem[];
  // As static variables, and with a base of the dynamic part that the compiler does not see through:
  // with these two laid over the staging area and a constant base, the same steps took 850 us instead
  // of 750 for 8192 bf16 tokens (D = 64: 178 and 157 us for 8 x 256 over 8192), and 1007 instead of
  // 959 for e4m3.
  __shared__ Line<kThreads> line;
  __shared__ Walk<P> walk;
  uint32_t sb = smem_u32(smem);
  asm volatile("" : "+r"(sb));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kBar + B_COUNT * 8);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kBar + B_COUNT * 8 + 4);
  // set when an aborted block could not confirm that its issued copies or MMAs have finished
  volatile int* unquiesced = reinterpret_cast<volatile int*>(smem + C::kBar + B_COUNT * 8 + 8);
  // unit v's is slot v % 4: when unit v + 4 is published, every warp has read unit v + 2 and so is
  // done with unit v
  int* nan_key = reinterpret_cast<int*>(smem + C::kBar + kNanKeyOff);
  auto bar = [&](int i) -> uint32_t { return sb + C::kBar + 8 * i; };
  int* err = a.c.status;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.x;
  let_next_start();
  wait_for_previous();
  if (threadIdx.x == 0) a.split[b].last = b;
  // (The first unit published in there, and what follows done before the wait: no faster for small
  // batches, and 1930 us instead of 1890 for 2048 tokens over 32768 e4m3 keys.)
  const Shares sh = begin_walk<P, kThreads>(a, line, b == 0,
                                            [&](Walk<P>& w, const Shares&, long long, long long) { walk = w; });
  if (b >= sh.blocks) return;
  // 128-byte-swizzled tiles need a 1024-byte aligned base; report, never fault
  if ((sb & 1023u) != 0) {
    if (threadIdx.x == 0) atomicCAS(err, 0, kErrSmemAlign);
    return;
  }

  Unit* unit_slot = reinterpret_cast<Unit*>(smem + C::kBar + kUnitOff);
  // consumer side: the unit of round v (valid = -1 when a wait gave up)
  auto next_unit = [&](int v, int code) -> Unit {
    Unit t;
    t.valid = -1;
    if (__all_sync(0xffffffffu, mbar_wait(bar(B_TFULL + (v & 1)), (v >> 1) & 1, abort_flag, err, code))) {
      const volatile Unit* src = unit_slot + (v & 1);
      t.valid = src->valid;
      t.i = src->i;
      t.a = src->a;
      t.n = src->n;
      t.len = src->len;
      t.h = src->h;
      t.u = src->u;
      t.kt0 = src->kt0;
      t.kt1 = src->kt1;
      t.slot = src->slot;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_TEMPTY + (v & 1)));
    }
    return t;
  };

  if (threadIdx.x == 0) {
    mbar_init(bar(B_QFULL), 1);
    mbar_init(bar(B_QEMPTY), 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(B_KFULL + s), kE4M3 ? 8 : 1);  // one arrival per 16 rows, or the copies' bytes
      mbar_init(bar(B_KEMPTY + s), 1);
      mbar_init(bar(B_VFULL + s), kE4M3 ? 8 : 1);
      mbar_init(bar(B_VEMPTY + s), 1);
      mbar_init(bar(B_SFULL + s), 1);
      mbar_init(bar(B_PFULL + 2 * s), 4);  // one arrival per softmax warp of the tile
      mbar_init(bar(B_PFULL + 2 * s + 1), 4);
      mbar_init(bar(B_ODONE + s), 1);
      mbar_init(bar(B_OFREE + s), 4);
      mbar_init(bar(B_TFULL + s), 1);
      mbar_init(bar(B_TEMPTY + s), 9 + (kE4M3 ? kLoaders : 0));
    }
    mbar_init(bar(B_DRAIN), 1);
    *abort_flag = 0;
    *unquiesced = 0;
    mbar_fence_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 8) {
    if constexpr (kE4M3) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp >= 10) {
      // ---------------------------------------------------------- loaders (e4m3)
      // The work is 16-row groups, each in one page: K's eight of a tile, V's eight, the next tile's.
      // They go round the six warps; the two that share their scheduler with no other loader take a
      // sixth turn in every 32. A warp fetches its next group as soon as it has handed one over, and
      // looks up the page of the one after (and only looks at it when its turn has come: a check at
      // once would wait for the lookup). Fetching row by row between a group's conversions instead, as
      // registers became free, put loads in front of the fence that hands the group over: 2048 tokens
      // over 32768 keys took 1980 us instead of 1920. A second group in flight, in registers, took 2515:
      // the code is twice as long and no longer stays in the instruction cache beside the softmax's;
      // in shared memory it took 2225, whose bandwidth the matrix instructions need.
      // A lane has 16 codes, two 16-byte pieces of bf16, of rows r0 + kStep x. Eight lanes store at a
      // time: four of an even and four of an odd row, whose swizzle puts them on different banks.
      constexpr int kLanes = D / 16, kStep = 32 / kLanes, kLoads = 16 / kStep;
      const int c = lane % kLanes, r0 = D == 128 ? (lane >> 3) ^ ((lane >> 2) & 1) : lane / kLanes;
      const int page_mask = (1 << a.c.page_shift) - 1;
      const int order = warp == 12 ? 0 : (warp == 13 ? 1 : (warp < 12 ? warp - 8 : warp - 10));
      int turn = 0;
      // from a group of this warp to its next: 32 groups are five rounds of six and two more
      auto step = [&]() -> int {
        const int last = order < 2 ? 5 : 4;
        const int d = turn < last ? 6 : (order < 2 ? 2 : 8);
        turn = turn < last ? turn + 1 : 0;
        return d;
      };
      bool ok = true;
      int J0 = 0;                            // key tiles before this unit
      int g1 = order, g2 = g1 + step();      // the group held, and the next
      for (int v = 0; ok; ++v) {
        const Unit t = next_unit(v, kErrPagedWait + 1);
        if (t.valid <= 0) break;
        const int* table = a.c.table + static_cast<long long>(t.i) * a.c.max_pages;
        const int g_end = (J0 + t.kt1 - t.kt0) * 16;
        auto first_key = [&](int g) -> int { return (t.kt0 + (g >> 4) - J0) * kTileN + 16 * (g & 7); };
        auto lookup = [&](int g) -> int {  // the block table's entry for group g; -1: nothing to read
          const int key0 = first_key(g);
          return g < g_end && key0 < t.len ? load(table + (key0 >> a.c.page_shift)) : -1;
        };
        uint4 raw[kLoads];  // of rows that are not there: anything
        const uint8_t* src = nullptr;
        int held = 0;        // rows r0 + kStep x with kStep x below it are there
        uint32_t byte = 0;   // lane l: scale of row l % 16; 256: not there
        auto fetch = [&](int g, int page) {
          const int key0 = first_key(g);
          const bool is_v = (g & 8) != 0, in = static_cast<unsigned>(page) < static_cast<unsigned>(a.c.n_pages);
          if (!in && g < g_end && key0 < t.len) atomicCAS(err, 0, kErrCachePage);
          const long long row = in ? page_row(a.c, page, t.h) + (key0 & page_mask) : 0;
          src = (is_v ? a.c.v_pages : a.c.k_pages) + (row + r0) * D + c * 16;
          held = in ? t.len - key0 - r0 : 0;
          byte = 256u;
          if (in && key0 + (lane & 15) < t.len) byte = load((is_v ? a.c.v_scales : a.c.k_scales) + row + (lane & 15));
#pragma unroll
          for (int x = 0; x < kLoads; ++x)
            if (kStep * x < held) raw[x] = load(reinterpret_cast<const uint4*>(src + kStep * x * D));
        };
#pragma unroll
        for (int x = 0; x < kLoads; ++x) raw[x] = make_uint4(0u, 0u, 0u, 0u);
        fetch(g1, lookup(g1));
        int page2 = lookup(g2);
        while (g1 < g_end) {
          const int J = g1 >> 4, s = J & 1;  // the block's key tile
          const bool is_v = (g1 & 8) != 0;
          ok = mbar_wait(bar((is_v ? B_VEMPTY : B_KEMPTY) + s), ((J >> 1) & 1) ^ 1, abort_flag, err, kErrPagedWait + 2);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          uint8_t* dst = smem + (is_v ? C::kV : C::kK) + s * C::kTileBytes + (16 * (g1 & 7) + r0) * 128;
          // Piece 2 c + y of row r0 + kStep x, swizzled by the row's last bits.
          auto piece = [&](int x, int y) -> uint4* {
            const int q = 2 * c + y;
            return reinterpret_cast<uint4*>(dst + (q >> 3) * kPanelBytes + kStep * x * 128 + (((q ^ (r0 + kStep * x)) & 7) << 4));
          };
          // A row's factor is 2^(byte - 127) * 2^120, in bf16 only up to a scale of 2^7. A group with a
          // larger one, or NaN, is done here, in two exact products; the code below then stores nothing.
          // (As branches of the loop below: 2047 us instead of 1913 for 2048 tokens over 32768 keys.)
          const uint32_t mine = byte;
          const bool large = __any_sync(0xffffffffu, mine - 135u <= 255u - 135u);
          if (large) {
            const uint32_t nan = __ballot_sync(0xffffffffu, is_v && mine == 255u);
            if (nan != 0u && lane == 0) atomicMin(nan_key + (v & 3), first_key(g1) + __ffs(nan) - 1);
            const bool none = mine == 256u || (nan >> lane & 1u);
            const uint32_t f2 = none || mine <= 134u ? 0x3f803f80u : (mine == 255u ? 0x7fc0u : (mine - 7u) << 7) * 0x10001u;
            const uint32_t f1 = none ? 0u : ((min(mine, 134u) + 120u) << 7) * 0x10001u;
#pragma unroll 1
            for (int x = 0; x < kLoads; ++x) {
              const uint32_t a1 = __shfl_sync(0xffffffffu, f1, r0 + kStep * x);
              const uint32_t a2 = __shfl_sync(0xffffffffu, f2, r0 + kStep * x);
#pragma unroll 1
              for (int y = 0; y < 2; ++y) {
                uint2 codes = make_uint2(0u, 0u);
                if (kStep * x < held) codes = load(reinterpret_cast<const uint2*>(src + kStep * x * D + 8 * y));
                uint32_t r[4];
                code_bits(codes, r);
                times(r, a1);
                times(r, a2);
                *piece(x, y) = make_uint4(r[0], r[1], r[2], r[3]);
              }
            }
          }
          const uint32_t f1 = mine == 256u ? 0u : ((mine + 120u) << 7) * 0x10001u;  // rows that are not there: zeros
#pragma unroll
          for (int x = 0; x < kLoads; ++x) {
            const uint32_t f = __shfl_sync(0xffffffffu, f1, r0 + kStep * x);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              uint32_t r[4];
              code_bits(y ? make_uint2(raw[x].z, raw[x].w) : make_uint2(raw[x].x, raw[x].y), r);
              times(r, f);
              if (!large) *piece(x, y) = make_uint4(r[0], r[1], r[2], r[3]);
            }
          }
          fence_proxy_async_smem();
          mbar_arrive_warp(bar((is_v ? B_VFULL : B_KFULL) + s));
          fetch(g2, page2);
          g1 = g2;
          g2 += step();
          page2 = lookup(g2);
        }
        J0 += t.kt1 - t.kt0;
      }
    } else if (warp == 8) {
      // ---------------------------------------------------------- walk, Q and (bf16) K, V loads
      // Lane 0 walks along the block's share and publishes each unit; then the lanes issue its
      // loads side by side: box j of Q, or page j of a key tile, is lane j's.
      if (lane == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmQ16);
        if constexpr (!kE4M3) {
          tma_prefetch_desc(&tmK);
          tma_prefetch_desc(&tmV);
        }
      }
      const long long w0 = sh.begin(b), w1 = sh.begin(b + 1);
      Walk<P> w = walk;
      bool more = true;
      bool ok = true;
      int J = 0;                                    // key tiles loaded
      int last_q = -1, last_kj = -1, last_vj = -1;  // round of the last Q load, tiles of the last K, V loads
      for (int v = 0; ok; ++v) {
        const int k = v & 1;
        ok = mbar_wait(bar(B_TEMPTY + k), ((v >> 1) & 1) ^ 1, abort_flag, err, kErrPagedWait + 3);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          if (v > 0) w.next(a, line, w1);
          int ga = 0, gb = 0;
          while ((more = more && w.i < a.c.n_seqs && w.f0 < w1)) {
            w.part(w0, w1, ga, gb);
            if (gb > ga) break;
            w.next(a, line, w1);  // the share has the group's overhead only
          }
          volatile Unit* dst = unit_slot + k;
          dst->valid = more ? 1 : 0;
          if constexpr (kE4M3) nan_key[v & 3] = INT32_MAX;
          if (more) {
            dst->i = w.i;
            dst->a = w.s.a;
            dst->n = w.s.n;
            dst->len = w.s.len;
            dst->h = w.h;
            dst->u = w.u;
            dst->kt0 = ga;
            dst->kt1 = gb;
            dst->slot = piece_slot(b, ga, gb, w.g);
            if (ga == 0 && gb < w.g) a.split[b] = SplitGroup{sh.owner(w.behind() - 1), w.s.a, w.s.n, w.h, w.u, {}};
          }
          mbar_arrive(bar(B_TFULL + k));
        }
        __syncwarp();
        const volatile Unit* src = unit_slot + k;  // stays until this unit's consumers have read it
        if (!src->valid) break;
        const SeqShape seq{src->a, src->n, src->len};
        const int h = src->h, kt0 = src->kt0, kt1 = src->kt1, x0 = 2 * src->u;
        const int* table = a.c.table + static_cast<long long>(src->i) * a.c.max_pages;
        ok = mbar_wait(bar(B_QEMPTY), (v & 1) ^ 1, abort_flag, err, kErrPagedWait + 4);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        {
          // Q: a tile of 128 tokens of one head is one box, others are boxes of 16 tokens of one
          // head; rows of boxes without a new token are never read for a stored row
          const ChunkRows::Shape z(seq, a.group);
          const int x = x0 + (lane >> 4), box = lane & 7, p = (lane >> 3) & 1;
          const ChunkRows::Tile tile = z.tile(x, a.group);
          const bool whole = tile.log_tokens == 7;
          int tok, head;
          const bool mine = p < C::kPanels && x < z.tiles && !(whole && box > 0) &&
                            tile.row(seq, a.group, box * kQBox, tok, head);
          const int large = __popc(__ballot_sync(0xffffffffu, mine && whole));
          const int small = __popc(__ballot_sync(0xffffffffu, mine && !whole));
          if (lane == 0) mbar_arrive_expect_tx(bar(B_QFULL), (large * kTileM + small * kQBox) * 128);
          __syncwarp();
          if (mine)
            tma_load_3d(sb + C::kQ + (x & 1) * C::kTileBytes + p * kPanelBytes + box * kQBox * 128, whole ? &tmQ : &tmQ16,
                        bar(B_QFULL), p * 64, seq.a + tok, h * a.group + head);
        }
        last_q = v;
        if constexpr (!kE4M3) {
          // A tile's pages, one to a lane; the next tile's are looked up while this one's loads go
          // out. Keys past the sequence and pages outside the cache take a box behind the last page,
          // which reads as zeros.
          const int rows = min(1 << a.c.page_shift, kTileN), n_boxes = kTileN / rows;
          auto lookup = [&](int kt) -> int {
            const int key = kt * kTileN + lane * rows;
            if (lane >= n_boxes || kt >= kt1 || key >= seq.len) return -1;
            const int page = load(table + (key >> a.c.page_shift));
            if (page >= 0 && page < a.c.n_pages) return page;
            atomicCAS(err, 0, kErrCachePage);
            return -1;
          };
          int page_next = lookup(kt0);
          for (int kt = kt0; kt < kt1 && ok; ++kt, ++J) {
            const int s = J & 1;
            const uint32_t ph = (J >> 1) & 1;
            const int outer = page_next < 0 ? max(a.c.n_pages * a.c.hkv, 1) : page_next * a.c.hkv + h;
            page_next = lookup(kt + 1);
            const int in_page = (kt * kTileN) & ((1 << a.c.page_shift) - 1);
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
              ok = ok && mbar_wait(bar((kv ? B_VEMPTY : B_KEMPTY) + s), ph ^ 1, abort_flag, err, kErrPagedWait + 2);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              const uint32_t full = bar((kv ? B_VFULL : B_KFULL) + s);
              if (lane == 0) mbar_arrive_expect_tx(full, C::kTileBytes);
              __syncwarp();
              if (lane < n_boxes) {
                const uint32_t to = sb + (kv ? C::kV : C::kK) + s * C::kTileBytes + lane * rows * 128;
#pragma unroll
                for (int p = 0; p < C::kPanels; ++p)
                  tma_load_3d(to + p * kPanelBytes, kv ? &tmV : &tmK, full, p * 64, in_page, outer);
              }
              if (kv) last_vj = J; else last_kj = J;
            }
          }
        }
      }
      if (lane == 0 && *abort_flag) {
        // an aborted block waits (bounded) for the loads that land in its shared memory; a stage is
        // loaded again only when its tile was consumed, so only the last two tiles' may be in flight
        bool done = last_q < 0 || mbar_wait_quiesce(bar(B_QFULL), last_q & 1, kWaitLimitNs);
        for (int j = max(last_kj - 1, 0); j <= last_kj; ++j)
          done = mbar_wait_quiesce(bar(B_KFULL + (j & 1)), (j >> 1) & 1, kWaitLimitNs) && done;
        for (int j = max(last_vj - 1, 0); j <= last_vj; ++j)
          done = mbar_wait_quiesce(bar(B_VFULL + (j & 1)), (j >> 1) & 1, kWaitLimitNs) && done;
        if (!done) *unquiesced = 1;
      }
    } else if (warp == 9) {
      // ---------------------------------------------------------- MMA issuer
      // the whole warp runs this with uniform operands; one elected lane issues each MMA/commit
      auto wwait = [&](uint32_t bb, uint32_t parity, int code) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(bb, parity, abort_flag, err, code));
      };
      auto issue_s = [&](int t, int s) {
        const uint32_t qbase = sb + C::kQ + t * C::kTileBytes;
        const uint32_t kbase = sb + C::kK + s * C::kTileBytes;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t o = (kk >> 2) * kPanelBytes + (kk & 3) * 32;
          mma_ss_w(tmem + t * 128, sdesc_sw128(qbase + o, 16, 1024), sdesc_sw128(kbase + o, 16, 1024), C::kIdescS, kk > 0);
        }
      };
      // tiles processed so far by each of the two softmax groups, and units: their barriers'
      // phases (a unit of one tile leaves group 1 out)
      int jt[2] = {0, 0}, ut[2] = {0, 0};
      // O_t += P_t V of the group's last issued S, in two halves of 64 keys
      auto issue_pv = [&](int t, int s, bool acc) -> bool {
        const uint32_t vbase = sb + C::kV + s * C::kTileBytes;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!wwait(bar(B_PFULL + 2 * t + half), (jt[t] - 1) & 1, kErrPagedWait + 5)) return false;
          tc_fence_after();
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4) {
            const int kk = 4 * half + k4;
            mma_ts_w(tmem + 256 + t * 128, tmem + t * 128 + kk * 8, sdesc_sw128(vbase + kk * 2048, kPanelBytes, 1024),
                     C::kIdescPV, (acc || kk > 0));
          }
        }
        return true;
      };
      bool ok = true;
      int J = 0;
      for (int v = 0; ok; ++v) {
        const Unit T = next_unit(v, kErrPagedWait + 6);
        if (T.valid <= 0) break;
        const int nt = P::tiles_of(SeqShape{T.a, T.n, T.len}, a.group, T.u);
        ok = wwait(bar(B_QFULL), v & 1, kErrPagedWait + 7);
        if (!ok) break;
        tc_fence_after();
        // PV of key tile J - 1 (the unit's jl - 1) for tile t; the first overwrites O_t, which the
        // previous unit's epilogue must have read out
        auto pv = [&](int t, int jl) -> bool {
          const int ps = (J - 1) & 1;
          if (t == 0) {
            if (!wwait(bar(B_VFULL + ps), ((J - 1) >> 1) & 1, kErrPagedWait + 8)) return false;
            if constexpr (!kE4M3) {
              // rows of the tile past the sequence, in its last page, become zeros
              const int held = T.len - (T.kt0 + jl - 1) * kTileN;
              if (held < kTileN) {
                for (int x = max(held, 0) * (D / 8) + lane; x < kTileN * (D / 8); x += 32) {
                  const int r = x / (D / 8), p = x % (D / 8);
                  *reinterpret_cast<uint4*>(smem + C::kV + ps * C::kTileBytes + (p >> 3) * kPanelBytes + r * 128 +
                                            (p & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                __syncwarp();
              }
            }
          }
          if (jl == 1 && ut[t] > 0 && !wwait(bar(B_OFREE + t), (ut[t] - 1) & 1, kErrPagedWait + 9)) return false;
          tc_fence_after();
          if (!issue_pv(t, ps, jl > 1)) return false;
          tc_commit_w(bar(B_ODONE + t));
          if (t == nt - 1) tc_commit_w(bar(B_VEMPTY + ps));
          return true;
        };
        int jl = 0;
        for (int kt = T.kt0; kt < T.kt1 && ok; ++kt, ++J, ++jl) {
          const int s = J & 1;
          if (!wwait(bar(B_KFULL + s), (J >> 1) & 1, kErrPagedWait + 10)) { ok = false; break; }
          tc_fence_after();
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!ok || t >= nt) break;
            if (jl > 0) ok = pv(t, jl);
            if (!ok) break;
            issue_s(t, s);
            tc_commit_w(bar(B_SFULL + t));
            ++jt[t];
          }
          if (ok) tc_commit_w(bar(B_KEMPTY + s));
        }
        if (!ok) break;
        // every S of this unit has been issued: Q is free once they complete
        tc_commit_w(bar(B_QEMPTY));
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (ok && t < nt) {
            ok = pv(t, jl);
            ++ut[t];
          }
      }
      // every issued MMA has completed once the drain barrier fires; wait for it also after an
      // abort, so that no MMA still reads shared memory or writes tensor memory when they are
      // released
      tc_commit_w(bar(B_DRAIN));
      if (!__all_sync(0xffffffffu, mbar_wait_quiesce(bar(B_DRAIN), 0, kWaitLimitNs)) && lane == 0) {
        *abort_flag = 1;
        *unquiesced = 1;
        atomicCAS(err, 0, kErrPagedWait + 11);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax (warps 0-7)
    if constexpr (kE4M3) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int t = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_addr = lane_base + t * 128;
    const uint32_t o_addr = lane_base + 256 + t * 128;
    bool ok = true;
    int J = 0;  // key tiles of this group
    for (int v = 0; ok; ++v) {
      const Unit T = next_unit(v, kErrPagedWait + 12);
      if (T.valid <= 0) break;
      const SeqShape seq{T.a, T.n, T.len};
      const ChunkRows::Shape z(seq, a.group);
      const int x = 2 * T.u + t;
      if (x >= z.tiles) continue;  // a unit of one tile
      const ChunkRows::Tile tile = z.tile(x, a.group);
      int tok, head;
      const bool mine = tile.row(seq, a.group, r, tok, head);
      const bool idle = !__any_sync(0xffffffffu, mine);  // a warp without a row keeps the barriers only
      // first key that this row does not see; rows that are not stored follow the fast path
      const int lim_row = !mine ? INT32_MAX : (a.causal ? max(0, T.len - T.n + tok + 1) : T.len);
      float m_used = -INFINITY;
      float l = 0.f;
      int jl = 0;
      for (int kt = T.kt0; kt < T.kt1; ++kt, ++J, ++jl) {
        ok = mbar_wait(bar(B_SFULL + t), J & 1, abort_flag, err, kErrPagedWait + 13);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (idle) {
          mbar_arrive_warp(bar(B_PFULL + 2 * t));
          mbar_arrive_warp(bar(B_PFULL + 2 * t + 1));
          continue;
        }
        const int lim = lim_row - kt * kTileN;  // visible key columns [0, lim)
        tc_fence_after();
        uint32_t sv[128];
        tmem_ld128(s_addr, sv);
        // columns that a row does not see become -inf, whose exp2 is 0 (most tiles have none)
        if (!__all_sync(0xffffffffu, lim >= kTileN)) {
#pragma unroll
          for (int e = 0; e < 128; ++e)
            if (e >= lim) sv[e] = 0xff800000u;
        }
        float mc[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          mc[c] = __uint_as_float(sv[32 * c]);
#pragma unroll
          for (int e = 0; e < 15; ++e)
            mc[c] = max3f(mc[c], __uint_as_float(sv[32 * c + 1 + 2 * e]), __uint_as_float(sv[32 * c + 2 + 2 * e]));
          mc[c] = fmaxf(mc[c], __uint_as_float(sv[32 * c + 31]));
        }
        const float mx = fmaxf(fmaxf(mc[0], mc[1]), fmaxf(mc[2], mc[3]));
        const float m_new = fmaxf(m_used, mx * a.scale_log2);
        float alpha = 1.f;
        const bool grow = m_new > m_used + kRescaleThreshold;
        if (grow) {
          alpha = fast_exp2(m_used - m_new);
          m_used = m_new;
        }
        const float mb = (m_used == -INFINITY) ? 0.f : m_used;
        // P (rounded to bf16: off by 2^-8 of itself at most) in two halves of 64 keys, each handed
        // to the MMA warp as soon as it is stored
        float rowsum = 0.f;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float2 acc2 = make_float2(0.f, 0.f);
#pragma unroll
          for (int c = 2 * half; c < 2 * half + 2; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int i0 = 32 * c + 2 * e;
              const float2 y = ffma2(__uint_as_float(sv[i0]), __uint_as_float(sv[i0 + 1]), a.scale_log2, a.scale_log2,
                                     -mb, -mb);
              const float p0 = fast_exp2(y.x), p1 = fast_exp2(y.y);
              acc2 = fadd2(acc2.x, acc2.y, p0, p1);
              pk[e] = pack_bf16(p0, p1);
            }
            tmem_st16(s_addr + c * 16, pk);
          }
          rowsum += acc2.x + acc2.y;
          if (half == 0) {
            // rows whose maximum grew are rescaled once PV of the key tile before is complete
            // (warp-uniform TMEM access)
            if (__any_sync(0xffffffffu, grow && jl > 0)) {
              ok = mbar_wait(bar(B_ODONE + t), (J - 1) & 1, abort_flag, err, kErrPagedWait + 14);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                uint32_t ov[32];
                tmem_ld32(o_addr + c * 32, ov);
#pragma unroll
                for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                tmem_st32(o_addr + c * 32, ov);
              }
            }
          }
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive_warp(bar(B_PFULL + 2 * t + half));
        }
        if (!ok) break;
        l = l * alpha + rowsum;
      }
      if (!ok) break;
      // epilogue: O_t is read out of TMEM (then released to the next unit's first PV) and stored:
      // normalised as bf16 when this block has the whole group, else as float32 sums for the merge
      ok = mbar_wait(bar(B_ODONE + t), (J - 1) & 1, abort_flag, err, kErrPagedWait + 15);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      if (idle) {
        tc_fence_before();
        mbar_arrive_warp(bar(B_OFREE + t));
        continue;
      }
      float inv = T.slot >= 0 ? 1.f : (l == 0.f ? 0.f : 1.f / l);
      // every V of the unit has been loaded: its last PV is complete
      const bool nan = kE4M3 && *const_cast<volatile int*>(nan_key + (v & 3)) < lim_row;
      if (nan) inv = __uint_as_float(0x7fc00000u);
      // The warp's rows go through a shared block of 32 rows x 128 bytes (16-byte slots XOR-swizzled
      // by row), 64 bf16 or 32 float32 channels at a time, so that stores write whole row segments:
      // lane l writes slot l % 8 of rows l / 8 + 4 i
      uint8_t* stg = smem + C::kStage + warp * 4096;
      const int wrow = (warp & 3) * 32, sub = lane >> 3, e8 = lane & 7;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t ov[32];
        tmem_ld32(o_addr + c * 32, ov);
        if (c == D / 32 - 1) {
          tc_fence_before();
          mbar_arrive_warp(bar(B_OFREE + t));
        }
        const bool wide = T.slot >= 0;  // 32 float32 channels fill the rows, 32 bf16 ones half of them
        if (wide || (c & 1) == 0) __syncwarp();  // the block has been read out
        if (wide) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<uint4*>(stg + lane * 128 + ((e ^ (lane & 7)) << 4)) =
                make_uint4(ov[4 * e], ov[4 * e + 1], ov[4 * e + 2], ov[4 * e + 3]);
          if (nan) {
#pragma unroll 1
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<uint4*>(stg + lane * 128 + (e << 4)) = make_uint4(0x7fc00000u, 0x7fc00000u, 0x7fc00000u, 0x7fc00000u);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint4 pk;
            pk.x = pack_bf16(__uint_as_float(ov[8 * e]) * inv, __uint_as_float(ov[8 * e + 1]) * inv);
            pk.y = pack_bf16(__uint_as_float(ov[8 * e + 2]) * inv, __uint_as_float(ov[8 * e + 3]) * inv);
            pk.z = pack_bf16(__uint_as_float(ov[8 * e + 4]) * inv, __uint_as_float(ov[8 * e + 5]) * inv);
            pk.w = pack_bf16(__uint_as_float(ov[8 * e + 6]) * inv, __uint_as_float(ov[8 * e + 7]) * inv);
            *reinterpret_cast<uint4*>(stg + lane * 128 + (((4 * (c & 1) + e) ^ (lane & 7)) << 4)) = pk;
          }
          if ((c & 1) == 0) continue;
        }
        __syncwarp();
#pragma unroll 2
        for (int i = 0; i < 8; ++i) {
          const int rr = 4 * i + sub, rt = wrow + rr;  // row of the warp, of the tile
          int tk, hd;
          if (!tile.row(seq, a.group, rt, tk, hd)) continue;
          const uint4 y = *reinterpret_cast<const uint4*>(stg + rr * 128 + ((e8 ^ (rr & 7)) << 4));
          if (wide)
            reinterpret_cast<uint4*>(a.part_o + (static_cast<long long>(T.slot) * P::kRows + t * kTileM + rt) * D)[c * 8 + e8] = y;
          else
            reinterpret_cast<uint4*>(a.o + (static_cast<long long>(T.h * a.group + hd) * a.c.total_new + T.a + tk) * D)[(c >> 1) * 8 + e8] = y;
        }
      }
      __syncwarp();  // the block is free for the next unit's epilogue
      if (mine) {
        if (T.slot >= 0)
          a.part_ml[static_cast<long long>(T.slot) * P::kRows + t * kTileM + r] = make_float2(m_used, l);
        else
          a.lse[static_cast<long long>(T.h * a.group + head) * a.c.total_new + T.a + tok] =
              l == 0.f ? -INFINITY : (m_used + log2f(l)) * 0.69314718055994531f;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*unquiesced) {
    // fallback only: an issued copy or MMA did not report completion within the wait limit
    const unsigned long long t0 = globaltimer();
    while (globaltimer() - t0 < 1000000ull) __nanosleep(1000);
  }
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool kE4M3>
fcp_status launch(AttnArgs a, void* workspace, int dev, int n_sm, int hq, cudaStream_t s) {
  using C = Cfg<D>;
  CUtensorMap mq, mq16, mk = {}, mv = {};
  if (const fcp_status st = make_bf16_map(&mq, a.q, hq, a.c.total_new, D, kTileM); st != FCP_OK) return st;
  if (const fcp_status st = make_bf16_map(&mq16, a.q, hq, a.c.total_new, D, kQBox); st != FCP_OK) return st;
  if constexpr (!kE4M3) {
    // pages and heads are the maps' outer dimension; a box is a page's rows, at most a tile
    const long long outer = static_cast<long long>(a.c.n_pages) * a.c.hkv;
    if (outer + a.c.hkv > INT32_MAX) return FCP_ERR_UNSUPPORTED;
    const int page = 1 << a.c.page_shift, n = static_cast<int>(std::max(outer, 1ll));
    fcp_status st;
    if ((st = make_bf16_map(&mk, a.c.k_pages, n, page, D, std::min(page, kTileN))) != FCP_OK) return st;
    if ((st = make_bf16_map(&mv, a.c.v_pages, n, page, D, std::min(page, kTileN))) != FCP_OK) return st;
  }
  // A bf16 cache's blocks come in clusters of two, of which only the placement is used: neighbours
  // on the line mostly read the same keys, and do so from one pair of SMs (4 sequences of 512 new
  // tokens over up to 16384 keys: 195 to 190 us; other shapes, and an e4m3 cache, within a percent or two either way).
  const int blocks = std::max(2, std::min(n_sm, kMaxChunkBlocks) & ~1);
  set_workspace<ChunkRows>(a, workspace, D, kMaxChunkBlocks);
  static std::atomic<uint64_t> allowed{0};
  if (const fcp_status st = allow_smem(chunk_kernel<D, kE4M3>, C::kSmemBytes, dev, allowed, "paged chunk smem attribute");
      st != FCP_OK)
    return st;
  if (const fcp_status st = launch_overlapped<kE4M3 ? 1 : 2>(chunk_kernel<D, kE4M3>, dim3(blocks), kThreads<kE4M3>, C::kSmemBytes, s,
                                              "paged chunk launch", mq, mq16, mk, mv, a);
      st != FCP_OK)
    return st;
  return launch_merge<ChunkRows, D>(a, blocks, 32, s);
}

}  // namespace

fcp_status launch_paged_chunk(const AttnArgs& a, int dtype, int d, int hq, void* workspace, int dev, int n_sm,
                              cudaStream_t s) {
  if (dtype == FCP_CACHE_E4M3)
    return d == 128 ? launch<128, true>(a, workspace, dev, n_sm, hq, s) : launch<64, true>(a, workspace, dev, n_sm, hq, s);
  return d == 128 ? launch<128, false>(a, workspace, dev, n_sm, hq, s) : launch<64, false>(a, workspace, dev, n_sm, hq, s);
}

}  // namespace fcp
