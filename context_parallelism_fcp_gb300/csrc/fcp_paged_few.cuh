// Shared by the kernels of few new rows (fcp_paged_few.cu, fcp_paged_few4.cu): copies, fragments and
// products of a warp, and a block's piece of the work.
#pragma once

#include "fcp_paged_sched.cuh"

namespace fcp {
namespace few {

constexpr int kWarps = 4;
constexpr int kFewThreads = kWarps * 32;
constexpr int kChunk = 16;                  // keys of the products' tiles, in one page
constexpr float kGrow = 8.0f;               // a row maximum is raised when it grows by over 2^8
constexpr float kUp = 7.0f;                 // f16: P starts at 2^7 and grows to 2^15, the top of f16

// Where piece c of row r lies in a tile. Rows of 128 bytes and more: 8 rows of one piece, and
// pieces 0-3 of two neighbouring rows, fall on different banks; rows of 64 bytes share a line
// of banks two by two, rows of 32 four by four.
template <int kRowBytes>
__device__ __forceinline__ int piece_at(int r, int c) {
  if constexpr (kRowBytes == 32) return r * 32 + ((c ^ ((r >> 2) & 1)) << 4);
  else if constexpr (kRowBytes == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
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

// The 8x8 matrix of 16-bit elements that the warp holds, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

struct Piece {
  int valid, i, h, u, a, n, len, end, ga, gb, slot;
};

}  // namespace few
}  // namespace fcp
