// The pages of a paged cache's sequences, kept on the GPU: sequences cut back to a length return
// their last whole pages to a stack of free ones, sequences that grow take pages from its top.
//
// admit: with p_i the pages that sequence i needs for its new tokens and r_i those tokens, both
// prefix sums over the sequences in order decide who is served, and place what is served: page k
// of sequence i is entry n_free - 1 - (p_0 + .. + p_(i-1)) - k of the stack, row j of it is packed row
// r_0 + .. + r_(i-1) + j. release: entry n_free + (freed by the sequences before) + k.
//
// Bound by latency: a step of a server touches a few KB. So it is one launch, in which every block
// adds up all sequences by itself (a few hundred are one load a thread) and then does 1024 packed
// rows (or table entries); nothing that a block reads is written until the last block has read it, and
// that one writes lengths, offsets and the stack's height. (128 sequences of a token each, released and
// admitted in two calls: 8.9 us, the host's time; with plain launches, which do not overlap the kernel before
// them, 10.2.) Rows find their sequence by a maximum scan
// over the block: each sequence marks its first row in the block.
#include <algorithm>

#include "fcp_paged.h"

namespace fcp {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kKeep = 2;  // sequences of a thread that are read once; more are read again in each pass

struct PoolArgs {
  int32_t* free_pages;
  int32_t* n_free;
  int32_t* lens;
  int32_t* table;
  int32_t* status;  // [0] the error, [1] blocks that are done, and 2^16 times those that report something
  int32_t n_pages, page_shift, n_seqs, max_pages;
};

__device__ __forceinline__ void report(const PoolArgs& p, int code) { atomicCAS(p.status, 0, code); }
__device__ __forceinline__ int pages_of(const PoolArgs& p, long long tokens) {
  return static_cast<int>((tokens + (1 << p.page_shift) - 1) >> p.page_shift);
}
__device__ __forceinline__ long long capacity(const PoolArgs& p) {
  return static_cast<long long>(p.max_pages) << p.page_shift;
}

// Sum of x over the threads before this one, and over all.
__device__ __forceinline__ long long scan(long long x, long long* warps, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  if (lane == 31) warps[warp] = y;
  __syncthreads();
  long long w = warps[lane], before = lane < warp ? w : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    w += __shfl_xor_sync(0xffffffffu, w, o);
  }
  total = w;
  __syncthreads();
  return before + y - x;
}

__device__ __forceinline__ int max_scan(int x, int* warps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x = max(x, z);
  }
  if (lane == 31) warps[warp] = x;
  __syncthreads();
  int before = lane < warp ? warps[lane] : -1;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) before = max(before, __shfl_xor_sync(0xffffffffu, before, o));
  __syncthreads();
  return max(x, before);
}

// Whether this block is the last to come here (its threads then see the others as done), and whether any block
// came with `found`, the same for all of its threads (they then see what the others wrote). The counter is left
// at zero.
__device__ __forceinline__ bool last_block(const PoolArgs& p, bool& found) {
  __shared__ int last, any;
  if (gridDim.x == 1) return true;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    const int before = atomicAdd(p.status + 1, found ? 0x10001 : 1);
    last = (before & 0xffff) == static_cast<int>(gridDim.x) - 1;
    any = found || (before >> 16) != 0;
    if (last) p.status[1] = 0;
    if (any) __threadfence();
  }
  __syncthreads();
  found = any != 0;
  return last != 0;
}

// The sequences of a thread: f(i, length, x[i]) in order. What does not fit a sequence's row is reported
// and has x = none.
struct Mine {
  int i0, i1, len[kKeep], x[kKeep];
  bool kept;
  const int32_t* from;
  __device__ __forceinline__ Mine(const PoolArgs& p, const int32_t* x_of) : from(x_of) {
    const int per = (p.n_seqs + kThreads - 1) / kThreads;
    i0 = min(static_cast<int>(threadIdx.x) * per, p.n_seqs);
    i1 = min(i0 + per, p.n_seqs);
    kept = per <= kKeep;
#pragma unroll
    for (int k = 0; k < kKeep; ++k)
      if (kept && i0 + k < i1) {
        len[k] = load(p.lens + i0 + k);
        x[k] = load(x_of + i0 + k);
      }
  }
  template <class F>
  __device__ __forceinline__ void each(const PoolArgs& p, F f) const {
    if (kept) {
#pragma unroll
      for (int k = 0; k < kKeep; ++k)
        if (i0 + k < i1) f(i0 + k, len[k], x[k]);
    } else {
      for (int i = i0; i < i1; ++i) f(i, load(p.lens + i), load(from + i));
    }
  }
};

struct Marks {
  long long warps[kWarps];
  int warp_max[kWarps];
  int seq[kThreads];    // -1: no sequence begins here
  int first[kThreads];  // row of the block where the sequence's rows begin: 0 or less
  int a[kThreads];      // the sequence's length, or its first freed page
  int b[kThreads];      // the stack's entries that those before it take
};

// A block does every gridDim.x-th 1024 rows.
__global__ void __launch_bounds__(kThreads) admit_kernel(const PoolArgs p, const int32_t* new_tokens, int total_new,
                                                         int32_t* cu, int32_t* granted, int32_t* positions,
                                                         long long* slots) {
  __shared__ Marks m;
  const int tid = threadIdx.x;
  let_next_start();
  wait_for_previous();
  const Mine mine(p, new_tokens);
  int n_free = load(p.n_free);
  const bool first_block = blockIdx.x == 0;
  if (n_free < 0 || n_free > p.n_pages) {
    if (first_block && tid == 0) report(p, kErrCacheBatch);
    n_free = 0;
  }
  // What a sequence wants and can have by itself: tokens and pages.
  auto asked = [&](int len, int x, int& pages) -> int {
    pages = 0;
    const bool ok = len >= 0 && len <= capacity(p) && x >= 0;
    if (!ok && first_block) report(p, kErrCacheBatch);
    if (!ok || x > capacity(p) - len) return 0;
    pages = pages_of(p, static_cast<long long>(len) + x) - pages_of(p, len);
    return x;
  };
  long long sum = 0, total;
  mine.each(p, [&](int, int len, int x) {
    int pages;
    asked(len, x, pages);
    sum += pages;
  });
  const long long pages0 = scan(sum, m.warps, total);
  long long at = pages0;
  sum = 0;
  mine.each(p, [&](int, int len, int x) {
    int pages;
    x = asked(len, x, pages);
    at += pages;
    sum += pages == 0 || at <= n_free ? x : 0;
  });
  const long long rows0 = scan(sum, m.warps, total);
  // f(i, length, tokens that it gets, pages of them, rows and pages before it)
  auto each = [&](auto f) {
    long long pg = pages0, row = rows0;
    mine.each(p, [&](int i, int len, int x) {
      int pages;
      x = asked(len, x, pages);
      const long long pg0 = pg, row0 = row;
      pg += pages;
      if (pages != 0 && pg > n_free) x = 0;
      row += x;
      if (row > total_new) x = 0;
      f(i, len, x, x > 0 ? pages : 0, row0, pg0);
    });
  };
  long long rows = 0, taken = 0;
  each([&](int, int, int x, int pages, long long row0, long long pg0) {
    if (x > 0) rows = row0 + x;
    if (x > 0 && pages > 0) taken = pg0 + pages;
  });
  // all rows and pages that are given: the largest, as the threads' sequences are in order
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    rows = max(rows, __shfl_xor_sync(0xffffffffu, rows, o));
    taken = max(taken, __shfl_xor_sync(0xffffffffu, taken, o));
  }
  if ((tid & 31) == 0) m.warps[tid >> 5] = rows << 32 | taken;  // both below 2^31
  __syncthreads();
  rows = m.warps[tid & 31] >> 32;
  taken = m.warps[tid & 31] & 0xffffffffll;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    rows = max(rows, __shfl_xor_sync(0xffffffffu, rows, o));
    taken = max(taken, __shfl_xor_sync(0xffffffffu, taken, o));
  }
  for (long long b0 = static_cast<long long>(blockIdx.x) * kThreads; b0 < total_new;
       b0 += static_cast<long long>(gridDim.x) * kThreads) {
    m.seq[tid] = -1;
    __syncthreads();
    each([&](int i, int len, int x, int, long long row0, long long pg0) {
      if (x > 0 && row0 < b0 + kThreads && row0 + x > b0) {
        const int y = static_cast<int>(max(row0 - b0, 0ll));
        m.seq[y] = i;
        m.first[y] = static_cast<int>(row0 - b0);
        m.a[y] = len;
        m.b[y] = static_cast<int>(pg0);
      }
    });
    __syncthreads();
    const int y = max_scan(m.seq[tid] >= 0 ? tid : -1, m.warp_max);
    const long long row = b0 + tid;
    if (row < total_new) {
      int pos = -1;
      long long slot = -1;
      if (y >= 0 && row < rows) {
        const int len = m.a[y], had = pages_of(p, len);
        pos = len + tid - m.first[y];
        const int k = pos >> p.page_shift, in = pos & ((1 << p.page_shift) - 1);
        int32_t* entry = p.table + static_cast<long long>(m.seq[y]) * p.max_pages + k;
        const int page = load(k < had ? entry : p.free_pages + (n_free - 1 - (m.b[y] + k - had)));
        if (k >= had && in == 0) *entry = page;  // every new page has its first position among the new rows
        if (page >= 0 && page < p.n_pages) slot = (static_cast<long long>(page) << p.page_shift) + in;
        else report(p, kErrCachePage);
      }
      if (positions) positions[row] = pos;
      if (slots) slots[row] = slot;
    }
    __syncthreads();
  }
  bool found = false;
  if (!last_block(p, found)) return;
  each([&](int i, int len, int x, int, long long row0, long long) {
    cu[i] = static_cast<int>(min(row0, rows));
    granted[i] = x;
    if (x > 0) p.lens[i] = len + x;
  });
  if (tid == 0) {
    cu[p.n_seqs] = static_cast<int>(rows);
    if (taken > 0) *p.n_free = n_free - static_cast<int>(taken);
  }
}

__global__ void __launch_bounds__(kThreads) release_kernel(const PoolArgs p, const int32_t* keep) {
  __shared__ Marks m;
  const int tid = threadIdx.x;
  let_next_start();
  wait_for_previous();
  const Mine mine(p, keep);
  const int n_free = load(p.n_free);
  const bool first_block = blockIdx.x == 0;
  // pages that a sequence gives back, the first of them in its row, and its new length
  auto given = [&](int len, int x, int& first, int& left) -> int {
    first = 0;
    left = len;
    if (len < 0 || len > capacity(p)) {
      if (first_block) report(p, kErrCacheBatch);
      return 0;
    }
    if (x >= 0 && x < len) left = x;
    first = pages_of(p, left);
    return pages_of(p, len) - first;
  };
  long long sum = 0, total;
  mine.each(p, [&](int, int len, int x) {
    int first, left;
    sum += given(len, x, first, left);
  });
  const long long before = scan(sum, m.warps, total);
  // a stack that is too high afterwards has pages twice: nothing is given back
  const bool fits = n_free >= 0 && n_free + total <= p.n_pages;
  if (!fits && first_block && tid == 0) report(p, kErrCacheBatch);
  bool lost = false;  // an id that is no page's was among those given back
  for (long long b0 = static_cast<long long>(blockIdx.x) * kThreads; fits && b0 < total;
       b0 += static_cast<long long>(gridDim.x) * kThreads) {
    m.seq[tid] = -1;
    __syncthreads();
    long long at = before;
    mine.each(p, [&](int i, int len, int x) {
      int first, left;
      const int n = given(len, x, first, left);
      if (n > 0 && at < b0 + kThreads && at + n > b0) {
        const int y = static_cast<int>(max(at - b0, 0ll));
        m.seq[y] = i;
        m.first[y] = static_cast<int>(at - b0);
        m.a[y] = first;
      }
      at += n;
    });
    __syncthreads();
    const int y = max_scan(m.seq[tid] >= 0 ? tid : -1, m.warp_max);
    if (b0 + tid < total) {
      int32_t* entry = p.table + static_cast<long long>(m.seq[y]) * p.max_pages + m.a[y] + (tid - m.first[y]);
      const int page = load(entry);
      if (page < 0 || page >= p.n_pages) {
        report(p, kErrCachePage);
        lost = true;
      }
      p.free_pages[n_free + b0 + tid] = page;
      *entry = -1;
    }
    lost = __syncthreads_or(lost) != 0;
  }
  if (!last_block(p, lost) || !fits) return;
  mine.each(p, [&](int i, int len, int x) {
    int first, left;
    given(len, x, first, left);
    if (left != len) p.lens[i] = left;
  });
  if (lost) {
    // It is left out of the stack: the others of this call move together, in order, 1 K at a time, which are
    // read before any of them is written over. (Past L1, which knows nothing of other blocks' writes.)
    int32_t* given_back = p.free_pages + n_free;
    long long kept = 0;
    for (long long b0 = 0; b0 < total; b0 += kThreads) {
      const int page = b0 + tid < total ? __ldcg(given_back + b0 + tid) : -1;
      const bool good = page >= 0 && page < p.n_pages;
      long long n;
      const long long at = kept + scan(good ? 1 : 0, m.warps, n);
      if (good) given_back[at] = page;
      kept += n;
    }
    total = kept;
  }
  if (tid == 0 && total > 0) *p.n_free = n_free + static_cast<int>(total);
}

fcp_status pool_args(const fcp_page_pool* c, PoolArgs* out) {
  if (c == nullptr) return FCP_ERR_INVALID;
  if (c->n_pages < 0 || c->page_size <= 0 || c->n_seqs < 0 || c->max_pages < 0) return FCP_ERR_INVALID;
  if (c->page_size < 16 || c->page_size > 4096 || (c->page_size & (c->page_size - 1)) != 0) return FCP_ERR_UNSUPPORTED;
  if (static_cast<long long>(c->max_pages) * c->page_size > 1ll << 30 || c->n_seqs > 65536) return FCP_ERR_UNSUPPORTED;
  if (!c->status || !aligned16(c->status) || !c->n_free || !aligned4(c->n_free)) return FCP_ERR_INVALID;
  if ((c->n_pages > 0 && !c->free_pages) || !aligned4(c->free_pages)) return FCP_ERR_INVALID;
  if (c->n_seqs > 0 && (!c->lens || (c->max_pages > 0 && !c->block_table))) return FCP_ERR_INVALID;
  if (!aligned4(c->lens) || !aligned4(c->block_table)) return FCP_ERR_INVALID;
  PoolArgs p;
  p.free_pages = c->free_pages;
  p.n_free = c->n_free;
  p.lens = c->lens;
  p.table = c->block_table;
  p.status = c->status;
  p.n_pages = c->n_pages;
  p.page_shift = 0;
  while ((1 << p.page_shift) < c->page_size) ++p.page_shift;
  p.n_seqs = c->n_seqs;
  p.max_pages = c->max_pages;
  *out = p;
  return FCP_OK;
}

}  // namespace
}  // namespace fcp

using namespace fcp;

extern "C" fcp_status fcp_pool_release(const fcp_page_pool* pool, const int32_t* keep, void* stream) {
  PoolArgs p;
  if (const fcp_status st = pool_args(pool, &p); st != FCP_OK) return st;
  if (p.n_seqs == 0) return FCP_OK;
  if (!keep || !aligned4(keep)) return FCP_ERR_INVALID;
  // How many entries go back only the GPU knows: a block for 8 K of the table's, which does them 1 K at a
  // time, and no more blocks than run at once.
  const long long entries = static_cast<long long>(p.n_seqs) * p.max_pages;
  int dev = 0, n_sm = 0;
  if (const fcp_status st = this_device(&dev, &n_sm); st != FCP_OK) return st;
  const unsigned blocks = static_cast<unsigned>(std::max(1ll, std::min<long long>((entries + 8191) / 8192, n_sm)));
  return launch_overlapped(release_kernel, dim3(blocks), kThreads, 0, static_cast<cudaStream_t>(stream),
                           "page pool release launch", p, keep);
}

extern "C" fcp_status fcp_pool_admit(const fcp_page_pool* pool, const int32_t* new_tokens, int32_t total_new,
                                     int32_t* cu_new, int32_t* granted, int32_t* positions, int64_t* slots,
                                     void* stream) {
  PoolArgs p;
  if (const fcp_status st = pool_args(pool, &p); st != FCP_OK) return st;
  if (total_new < 0) return FCP_ERR_INVALID;
  if (total_new > 1 << 30) return FCP_ERR_UNSUPPORTED;
  if (!cu_new || !aligned4(cu_new) || !aligned4(positions) || (reinterpret_cast<uintptr_t>(slots) & 7u) != 0)
    return FCP_ERR_INVALID;
  if (p.n_seqs > 0 && (!new_tokens || !granted || !aligned4(new_tokens) || !aligned4(granted) || new_tokens == granted))
    return FCP_ERR_INVALID;
  int dev = 0, n_sm = 0;
  if (const fcp_status st = this_device(&dev, &n_sm); st != FCP_OK) return st;
  // a block for 1 K rows, and no more blocks than run at once: each adds all sequences up (354000 rows of 300
  // sequences, released and admitted: 17.9 us with a block for each 1 K rows, 12.6 so)
  const unsigned blocks = static_cast<unsigned>(std::max(1, std::min((total_new + kThreads - 1) / kThreads, n_sm)));
  return launch_overlapped(admit_kernel, dim3(blocks), kThreads, 0, static_cast<cudaStream_t>(stream),
                           "page pool admit launch", p, new_tokens, static_cast<int>(total_new), cu_new, granted, positions,
                           reinterpret_cast<long long*>(slots));
}
