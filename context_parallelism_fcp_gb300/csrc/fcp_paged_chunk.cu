// Attention of chunks of new tokens over a paged cache on sm_103a (tcgen05 + TMEM).
//
// A unit is up to two tiles of 128 rows of one KV head. A tile is 2^t new tokens (16, 32, 64 or
// 128, by the sequence's new tokens) times 128 / 2^t query heads of the group, head by head, so
// that short chunks fill the tile with heads instead of padding, and every key tile loaded
// serves all of a unit's rows. Rows are computed independently of one another: those past the
// chunk or the group hold whatever is in shared memory and are not stored.
//
// As in the forward over a work list, S_t = Q_t K^T and O_t += P_t V run on the tensor core
// with accumulators in tensor memory while the other tile's softmax runs; what differs is where
// keys come from. A key tile is 128 positions, gathered from their pages by four loader warps
// into the 128-byte-swizzled layout that the matrix instructions read: as asynchronous copies
// for bf16, and for e4m3 through registers, where each row is scaled by its power of two. That
// product is exact, so the kernel computes the attention over what reading the cache gives, and
// the tensor core runs the same bf16 instructions for both. Rows past the sequence become zeros,
// since a zero weight times NaN is NaN.
//
// 16 warps: 0-3 and 4-7 softmax of tile 0 and 1 (thread = row = TMEM lane), 8 the walk along
// the block's share of the work and Q's TMA loads, 9 MMA, 12-15 loaders. TMEM columns: S_t at
// [128 t, 128 t + 128), overwritten by P_t as bf16; O_t at [256 + 128 t, 256 + 128 t + D).
#include <algorithm>
#include <cmath>

#include "fcp_paged_sched.cuh"

namespace fcp {
namespace {

using namespace dev;

constexpr int kThreads = 512;
constexpr int kPanelBytes = kTileM * 128;  // 128 rows x 64 bf16 channels
constexpr float kRescaleThreshold = 8.0f;   // log2 units
constexpr int kQBox = 16;                   // tokens of one TMA load of Q
// registers a thread: the launch gives 128; softmax warps take what the others leave
constexpr int kRegsSoftmax = 176, kRegsControl = 64, kRegsLoader = 96;
static_assert(2 * kRegsSoftmax + kRegsControl + kRegsLoader <= 4 * 128, "the split fits the launch's registers");

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
  B_TEMPTY = 23,  // 2 slots: 13 warps (MMA, softmax, loaders) have read it
  B_COUNT = 25
};

// A block's piece of a group: key tiles [kt0, kt1) of unit u.
struct Unit {
  int valid, i, a, n, len, h, u, kt0, kt1, slot, pad0, pad1;
};
constexpr int kUnitOff = 256;
constexpr int kBarArea = kUnitOff + 2 * static_cast<int>(sizeof(Unit));
static_assert(B_COUNT * 8 + 12 <= kUnitOff, "barrier area");

template <int D>
struct Cfg {
  static constexpr int kTileBytes = kTileM * D * 2;
  static constexpr int kPanels = D / 64;
  static constexpr int kQ = 0;                     // 2 tiles
  static constexpr int kK = 2 * kTileBytes;        // 2 stages
  static constexpr int kV = 4 * kTileBytes;        // 2 stages
  static constexpr int kBar = 6 * kTileBytes;
  static constexpr int kStage = kBar + kBarArea;   // epilogue: [32 rows][32 float32] per softmax warp
  static constexpr int kStageBytes = 8 * 32 * 32 * 4;
  static constexpr int kEnd = kStage + kStageBytes;
  // at least half the SM's shared memory, so one block per SM holds all 512 TMEM columns
  static constexpr int kSmemBytes = kEnd > 118 * 1024 ? kEnd : 118 * 1024;
  static_assert(kStage % 16 == 0, "16-byte aligned staging");
  static_assert(kSmemBytes <= 232448, "shared memory per block");
  static constexpr uint32_t kIdescS = idesc_bf16(kTileM, kTileN, false, false);
  static constexpr uint32_t kIdescPV = idesc_bf16(kTileM, D, false, true);
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool fill) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(fill ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

// 16 codes and their row's scale byte as 16 bf16 channels: code * 2^(byte - 127). The code's bits
// in bf16's fields are code * 2^-120, and 2^120 is taken into the scale where bf16 holds the
// product of both; larger scales take two exact products.
__device__ __forceinline__ void scaled16(const uint4 x, uint32_t byte, uint4& lo, uint4& hi) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t r[8];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t y = __byte_perm(w[i], 0, j ? 0x3424 : 0x1404);
      r[2 * i + j] = (y & 0x80008000u) | ((y & 0x7f007f00u) >> 4);
    }
  auto times = [&](uint32_t f) {
    f |= f << 16;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __nv_bfloat162 y =
          __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&r[i]), *reinterpret_cast<const __nv_bfloat162*>(&f));
      r[i] = *reinterpret_cast<const uint32_t*>(&y);
    }
  };
  if (byte <= 134u) {
    times((byte + 120u) << 7);
  } else {
    times(254u << 7);
    times(byte == 255u ? 0x7fc0u : (byte - 7u) << 7);
  }
  lo = make_uint4(r[0], r[1], r[2], r[3]);
  hi = make_uint4(r[4], r[5], r[6], r[7]);
}

template <int D, bool kE4M3>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap tmQ, const AttnArgs a) {
  using C = Cfg<D>;
  using P = ChunkRows;
  extern __shared__ __align__(1024) uint8_t smem[];
  // the line lies where the first epilogue writes, long after the walk has been placed on it
  Line<kThreads>& line = *reinterpret_cast<Line<kThreads>*>(smem + C::kStage);
  static_assert(sizeof(Line<kThreads>) <= C::kStageBytes, "the line fits the epilogue's staging");
  const uint32_t sb = smem_u32(smem);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kBar + B_COUNT * 8);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kBar + B_COUNT * 8 + 4);
  // set when an aborted block could not confirm that its issued copies or MMAs have finished
  volatile int* unquiesced = reinterpret_cast<volatile int*>(smem + C::kBar + B_COUNT * 8 + 8);
  auto bar = [&](int i) -> uint32_t { return sb + C::kBar + 8 * i; };
  int* err = a.c.status;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.x;
  if (threadIdx.x == 0) a.split[b].last = b;
  build_line<P, kThreads>(a, line, b == 0);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Shares sh(line.prefix[kThreads], gridDim.x);
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
      mbar_init(bar(B_KFULL + s), 4);  // one arrival per loader warp
      mbar_init(bar(B_KEMPTY + s), 1);
      mbar_init(bar(B_VFULL + s), 4);
      mbar_init(bar(B_VEMPTY + s), 1);
      mbar_init(bar(B_SFULL + s), 1);
      mbar_init(bar(B_PFULL + 2 * s), 4);  // one arrival per softmax warp of the tile
      mbar_init(bar(B_PFULL + 2 * s + 1), 4);
      mbar_init(bar(B_ODONE + s), 1);
      mbar_init(bar(B_OFREE + s), 4);
      mbar_init(bar(B_TFULL + s), 1);
      mbar_init(bar(B_TEMPTY + s), 13);
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

  if (warp >= 12) {
    // ------------------------------------------------------------ loaders
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLoader));
    const int tid = threadIdx.x - 12 * 32;
    constexpr int kLanes = kE4M3 ? D / 16 : D / 8;  // threads to a row, 16 bytes of it each
    constexpr int kRowsAtOnce = 128 / kLanes;
    constexpr int kPasses = kTileN / kRowsAtOnce;
    const int r0 = tid / kLanes, c = tid % kLanes;
    // 16-byte piece p of row r of a tile: 128-byte rows of 64-channel panels, XOR-swizzled by r & 7
    // (r = r0 + a multiple of 8, so the swizzle is the thread's own)
    auto piece = [&](int p) -> uint32_t { return (p >> 3) * kPanelBytes + r0 * 128 + (((p & 7) ^ (r0 & 7)) << 4); };
    const int page_mask = (1 << a.c.page_shift) - 1;
    bool ok = true;
    int J = 0;
    int pending = -1;  // barrier of the copies that are in flight and not signalled
    auto signal = [&]() {
      if (pending >= 0) {
        fence_proxy_async_smem();
        mbar_arrive_warp(bar(pending));
      }
    };
    for (int v = 0; ok; ++v) {
      const Unit t = next_unit(v, kErrPagedWait + 1);
      if (t.valid <= 0) break;
      const int* table = a.c.table + static_cast<long long>(t.i) * a.c.max_pages;
      // lane l < 8 looks up the page of the tile's keys [16 l, 16 l + 16); -1: nothing to read
      auto lookup = [&](int kt) -> int {
        const int key = kt * kTileN + 16 * (lane & 7);
        if (kt >= t.kt1 || key >= t.len) return -1;
        const int pg = __ldg(table + (key >> a.c.page_shift));
        if (pg < 0 || pg >= a.c.n_pages) {
          atomicCAS(err, 0, kErrCachePage);
          return -1;
        }
        return pg;
      };
      int page_next = lookup(t.kt0);
      // pass x of key tile kt: its row of the cache; false for rows that become zeros
      auto row_of = [&](int page, int kt, int x, long long& row) -> bool {
        const int pg = __shfl_sync(0xffffffffu, page, (x * kRowsAtOnce + (kRowsAtOnce > 16 ? r0 & 16 : 0)) >> 4);
        const int key = kt * kTileN + r0 + x * kRowsAtOnce;
        row = page_row(a.c, pg, t.h) + (key & page_mask);
        return key < t.len && pg >= 0;
      };
      if constexpr (!kE4M3) {
        const uint32_t off = piece(c);
        for (int kt = t.kt0; kt < t.kt1 && ok; ++kt, ++J) {
          const int page = page_next;
          page_next = lookup(kt + 1);
          const int s = J & 1;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            ok = ok && mbar_wait(bar((kv ? B_VEMPTY : B_KEMPTY) + s), ((J >> 1) & 1) ^ 1, abort_flag, err, kErrPagedWait + 2);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint8_t* pages = kv ? a.c.v_pages : a.c.k_pages;
            const uint32_t dst = sb + (kv ? C::kV : C::kK) + s * C::kTileBytes + off;
#pragma unroll
            for (int x = 0; x < kPasses; ++x) {
              long long row;
              const bool on = row_of(page, kt, x, row);
              cp_async16(dst + x * kRowsAtOnce * 128, pages + (on ? row * (2 * D) + c * 16 : 0), on);
            }
            cp_commit();
            cp_wait<1>();  // the copies before these have arrived: theirs is the tile to hand over
            signal();
            pending = (kv ? B_VFULL : B_KFULL) + s;
          }
        }
      } else {
        // The codes of a half step (K or V of a tile) are loaded while the half step before is
        // turned into bf16: as soon as a register is converted, its next load goes out.
        uint4 raw[kPasses];
        uint32_t byte[kPasses];
        auto load = [&](int page, int kt, int kv, int x) {
          long long row;
          const bool on = row_of(page, kt, x, row);
          raw[x] = make_uint4(0u, 0u, 0u, 0u);
          byte[x] = 127u;
          if (on) {
            raw[x] = __ldg(reinterpret_cast<const uint4*>((kv ? a.c.v_pages : a.c.k_pages) + row * D) + c);
            byte[x] = __ldg((kv ? a.c.v_scales : a.c.k_scales) + row);
          }
        };
        // lanes of the row's other panel store their two pieces in the other order, so that the
        // eight lanes of a row always hit different banks
        const uint32_t swap = (c >> 2) & 1;
        const uint32_t off0 = piece(2 * c + swap), off1 = piece(2 * c + 1 - swap);
#pragma unroll
        for (int x = 0; x < kPasses; ++x) load(page_next, t.kt0, 0, x);
        for (int kt = t.kt0; kt < t.kt1 && ok; ++kt, ++J) {
          const int page = page_next;
          page_next = lookup(kt + 1);
          const int s = J & 1;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            ok = ok && mbar_wait(bar((kv ? B_VEMPTY : B_KEMPTY) + s), ((J >> 1) & 1) ^ 1, abort_flag, err, kErrPagedWait + 2);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            uint8_t* dst = smem + (kv ? C::kV : C::kK) + s * C::kTileBytes;
#pragma unroll
            for (int x = 0; x < kPasses; ++x) {
              const uint4 y = raw[x];
              const uint32_t f = byte[x];
              load(kv ? page_next : page, kt + kv, 1 - kv, x);
              uint4 lo, hi;
              scaled16(y, f, lo, hi);
              *reinterpret_cast<uint4*>(dst + off0 + x * kRowsAtOnce * 128) = swap ? hi : lo;
              *reinterpret_cast<uint4*>(dst + off1 + x * kRowsAtOnce * 128) = swap ? lo : hi;
            }
            fence_proxy_async_smem();
            mbar_arrive_warp(bar((kv ? B_VFULL : B_KFULL) + s));
          }
        }
      }
    }
    cp_wait<0>();
    if (ok) signal();
  } else if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    if (warp == 8) {
      // ---------------------------------------------------------- walk and Q producer
      if (lane == 0) {
        tma_prefetch_desc(&tmQ);
        const long long w0 = sh.begin(b), w1 = sh.begin(b + 1);
        Walk<P> w;
        bool more = seek<P, kThreads>(a, line, w0, w);
        int last_q = -1;  // round of the last Q load
        for (int v = 0;; ++v) {
          const int k = v & 1;
          if (!mbar_wait(bar(B_TEMPTY + k), ((v >> 1) & 1) ^ 1, abort_flag, err, kErrPagedWait + 3)) break;
          if (v > 0) w.next(a);
          more = more && w.i < a.c.n_seqs && w.f0 < w1;
          volatile Unit* dst = unit_slot + k;
          dst->valid = more ? 1 : 0;
          if (more) {
            const int ga = static_cast<int>(max(w0 - w.f0, 0ll));
            const int gb = static_cast<int>(min(w1 - w.f0, static_cast<long long>(w.g)));
            dst->i = w.i;
            dst->a = w.s.a;
            dst->n = w.s.n;
            dst->len = w.s.len;
            dst->h = w.h;
            dst->u = w.u;
            dst->kt0 = ga;
            dst->kt1 = gb;
            dst->slot = piece_slot(b, ga, gb, w.g);
            if (ga == 0 && gb < w.g) a.split[b] = SplitGroup{sh.owner(w.f0 + w.g - 1), w.s.a, w.s.n, w.h, w.u, {}};
          }
          mbar_arrive(bar(B_TFULL + k));
          if (!more) break;
          if (!mbar_wait(bar(B_QEMPTY), (v & 1) ^ 1, abort_flag, err, kErrPagedWait + 4)) break;
          // Q: boxes of 16 tokens of one head; the rest of the tiles is never read for a stored row
          const ChunkRows::Shape z(w.s, a.group);
          const int x1 = min(2 * w.u + 2, z.tiles);
          for (int pass = 0; pass < 2; ++pass) {
            int boxes = 0;
            for (int x = 2 * w.u; x < x1; ++x) {
              const int tok0 = (x / z.head_tiles) << z.log_tokens, head0 = (x % z.head_tiles) * z.heads;
              const int heads = min(z.heads, a.group - head0);
              const int toks = min((1 << z.log_tokens), w.s.n - tok0);
              if (pass == 0) {
                boxes += heads * ((toks + kQBox - 1) / kQBox);
                continue;
              }
              for (int hh = 0; hh < heads; ++hh)
                for (int tok = 0; tok < toks; tok += kQBox)
                  for (int p = 0; p < C::kPanels; ++p)
                    tma_load_3d(sb + C::kQ + (x & 1) * C::kTileBytes + p * kPanelBytes +
                                    ((hh << z.log_tokens) + tok) * 128,
                                &tmQ, bar(B_QFULL), p * 64, w.s.a + tok0 + tok, w.h * a.group + head0 + hh);
            }
            if (pass == 0) mbar_arrive_expect_tx(bar(B_QFULL), boxes * kQBox * 128 * C::kPanels);
          }
          last_q = v;
        }
        // an aborted block waits (bounded) for the loads that land in its shared memory
        if (*abort_flag && last_q >= 0 && !mbar_wait_quiesce(bar(B_QFULL), last_q & 1, kWaitLimitNs)) *unquiesced = 1;
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
          if (t == 0 && !wwait(bar(B_VFULL + ps), ((J - 1) >> 1) & 1, kErrPagedWait + 8)) return false;
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
          for (int t = 0; t < nt; ++t) {
            if (jl > 0 && !pv(t, jl)) { ok = false; break; }
            issue_s(t, s);
            tc_commit_w(bar(B_SFULL + t));
            ++jt[t];
          }
          if (ok) tc_commit_w(bar(B_KEMPTY + s));
        }
        if (!ok) break;
        // every S of this unit has been issued: Q is free once they complete
        tc_commit_w(bar(B_QEMPTY));
        for (int t = 0; t < nt && ok; ++t) ok = pv(t, jl);
        for (int t = 0; t < nt; ++t) ++ut[t];
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
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
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
      const int tok0 = (x / z.head_tiles) << z.log_tokens, head0 = (x % z.head_tiles) * z.heads;
      const int tok = tok0 + (r & ((1 << z.log_tokens) - 1)), head = head0 + (r >> z.log_tokens);
      const bool mine = tok < T.n && head < a.group;
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
        // tiles with every column visible to every row of the warp take the short path
        const bool full = __all_sync(0xffffffffu, lim >= kTileN);
        float mx;
        if (full) {
          float mc[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            mc[c] = __uint_as_float(sv[32 * c]);
#pragma unroll
            for (int e = 0; e < 15; ++e)
              mc[c] = max3f(mc[c], __uint_as_float(sv[32 * c + 1 + 2 * e]), __uint_as_float(sv[32 * c + 2 + 2 * e]));
            mc[c] = fmaxf(mc[c], __uint_as_float(sv[32 * c + 31]));
          }
          mx = fmaxf(fmaxf(mc[0], mc[1]), fmaxf(mc[2], mc[3]));
        } else {
          mx = -INFINITY;
#pragma unroll
          for (int e = 0; e < 128; ++e)
            if (e < lim) mx = fmaxf(mx, __uint_as_float(sv[e]));
        }
        const float m_new = fmaxf(m_used, mx * a.scale_log2);
        float alpha = 1.f;
        const bool grow = m_new > m_used + kRescaleThreshold;
        if (grow) {
          alpha = fast_exp2(m_used - m_new);
          m_used = m_new;
        }
        const float mb = (m_used == -INFINITY) ? 0.f : m_used;
        // P (rounded to bf16: off by 2^-9 of itself at most) in two halves of 64 keys, each handed
        // to the MMA warp as soon as it is stored
        float rowsum = 0.f;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (full) {
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
          } else {
#pragma unroll
            for (int c = 2 * half; c < 2 * half + 2; ++c) {
              uint32_t pk[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const int c0 = c * 32 + 2 * e;
                const float p0 = (c0 < lim) ? fast_exp2(fmaf(__uint_as_float(sv[c0]), a.scale_log2, -mb)) : 0.f;
                const float p1 = (c0 + 1 < lim) ? fast_exp2(fmaf(__uint_as_float(sv[c0 + 1]), a.scale_log2, -mb)) : 0.f;
                rowsum += p0 + p1;
                pk[e] = pack_bf16(p0, p1);
              }
              tmem_st16(s_addr + c * 16, pk);
            }
          }
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
      const float inv = T.slot >= 0 ? 1.f : (l == 0.f ? 0.f : 1.f / l);
      // Each 32-column slice of the warp's rows goes through a shared [32][32] float32 block
      // (16-byte slots XOR-swizzled by row), so that stores write whole row segments
      float4* stg = reinterpret_cast<float4*>(smem + C::kStage + warp * 4096);
      auto place = [&](int rr, int& tk, int& hd) -> bool {  // row rr of the tile
        tk = tok0 + (rr & ((1 << z.log_tokens) - 1));
        hd = head0 + (rr >> z.log_tokens);
        return tk < T.n && hd < a.group;
      };
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t ov[32];
        tmem_ld32(o_addr + c * 32, ov);
        if (c == D / 32 - 1) {
          tc_fence_before();
          mbar_arrive_warp(bar(B_OFREE + t));
        }
        if (c > 0) __syncwarp();  // the previous slice has been read out of the block
#pragma unroll
        for (int e = 0; e < 8; ++e)
          stg[lane * 8 + (e ^ (lane & 7))] =
              make_float4(__uint_as_float(ov[4 * e]) * inv, __uint_as_float(ov[4 * e + 1]) * inv,
                          __uint_as_float(ov[4 * e + 2]) * inv, __uint_as_float(ov[4 * e + 3]) * inv);
        __syncwarp();
        const int wrow = (warp & 3) * 32;
        if (T.slot >= 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rr = 4 * i + (lane >> 3), e = lane & 7;
            int tk, hd;
            if (place(wrow + rr, tk, hd)) {
              const long long at = static_cast<long long>(T.slot) * P::kRows + t * kTileM + wrow + rr;
              reinterpret_cast<float4*>(a.part_o + at * D)[c * 8 + e] = stg[rr * 8 + (e ^ (rr & 7))];
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int rr = 8 * i + (lane >> 2), e = lane & 3;
            int tk, hd;
            if (place(wrow + rr, tk, hd)) {
              const float4 y0 = stg[rr * 8 + ((2 * e) ^ (rr & 7))], y1 = stg[rr * 8 + ((2 * e + 1) ^ (rr & 7))];
              const long long at = static_cast<long long>(T.h * a.group + hd) * a.c.total_new + T.a + tk;
              uint4 pk;
              pk.x = pack_bf16(y0.x, y0.y);
              pk.y = pack_bf16(y0.z, y0.w);
              pk.z = pack_bf16(y1.x, y1.y);
              pk.w = pack_bf16(y1.z, y1.w);
              reinterpret_cast<uint4*>(a.o + at * D + c * 32)[e] = pk;
            }
          }
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
fcp_status launch(AttnArgs a, void* workspace, int n_sm, int hq, cudaStream_t s) {
  using C = Cfg<D>;
  CUtensorMap mq;
  if (const fcp_status st = make_bf16_map(&mq, a.q, hq, a.c.total_new, D, kQBox); st != FCP_OK) return st;
  const int blocks = std::min(n_sm, kMaxChunkBlocks);
  set_workspace<ChunkRows>(a, workspace, D, kMaxChunkBlocks);
  FCP_CUDA_TRY(cudaFuncSetAttribute(chunk_kernel<D, kE4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes),
               "paged chunk smem attribute");
  chunk_kernel<D, kE4M3><<<blocks, kThreads, C::kSmemBytes, s>>>(mq, a);
  FCP_CUDA_TRY(cudaGetLastError(), "paged chunk launch");
  return launch_merge<ChunkRows, D>(a, blocks, 32, s);
}

}  // namespace

fcp_status launch_paged_chunk(const AttnArgs& a, int dtype, int d, int hq, void* workspace, int n_sm, cudaStream_t s) {
  if (dtype == FCP_CACHE_E4M3)
    return d == 128 ? launch<128, true>(a, workspace, n_sm, hq, s) : launch<64, true>(a, workspace, n_sm, hq, s);
  return d == 128 ? launch<128, false>(a, workspace, n_sm, hq, s) : launch<64, false>(a, workspace, n_sm, hq, s);
}

}  // namespace fcp
