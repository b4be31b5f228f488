// Pieces of the kernels in which each warp streams weight rows straight from
// global memory into warp-wide matrix instructions (m16n8k16, 16-bit operands,
// fp32 sums): asynchronous 16-byte copies into a queue of the lane's own, the
// instruction, and exact conversions of 8- and 4-bit weights to 16 bits.
//
// Lane (g, t) = (lane / 4, lane % 4) of an m16n8k16 holds, of A (16 weight
// rows) rows g and g + 8 and of B (8 activation rows) row g, two pairs of
// neighbouring values along K.  Which values along K those are is free, as
// long as A and B agree for each t: a lane takes 16 contiguous bytes of its
// rows, and all of them are operands of that lane, so nothing is exchanged
// between lanes and nothing is rearranged in shared memory.
#pragma once

#include "common.cuh"

namespace oes {

// 16 bytes global -> shared past L1, zeros instead where `take` is false (the
// source is not read then)
__device__ __forceinline__ void cp_async16_take(uint32_t dst_smem, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst_smem), "l"(src), "r"(take ? 16 : 0)
               : "memory");
}
// the first n <= 16 bytes, zeros behind them
__device__ __forceinline__ void cp_async16_part(uint32_t dst_smem, const void* src, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst_smem), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async4_take(uint32_t dst_smem, const void* src, bool take) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst_smem), "l"(src), "r"(take ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// waits until at most N of this thread's committed groups are in flight
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// D (+)= A B^T: a0, a2 row g; a1, a3 row g + 8; b0, b1 column g; d[0], d[1] are
// row g, columns 2t and 2t + 1, d[2], d[3] row g + 8.  FRESH: from zero.
template <bool F16, bool FRESH = false>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  const float c0 = FRESH ? 0.0f : d[0], c1 = FRESH ? 0.0f : d[1], c2 = FRESH ? 0.0f : d[2], c3 = FRESH ? 0.0f : d[3];
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// two e4m3 codes (low byte first) -> f16x2, exact
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two) {
  uint32_t r;
  asm("{ .reg .b16 h; cvt.u16.u32 h, %1; cvt.rn.f16x2.e4m3x2 %0, h; }" : "=r"(r) : "r"(two));
  return r;
}
// four e4m3 codes -> two f16x2, exact; NaN stays NaN
__device__ __forceinline__ void e4m3x4_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{ .reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b; }"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
// eight e2m1 codes (element 2i in the low nibble of byte i) -> four f16x2, exact
__device__ __forceinline__ void e2m1x8_f16x8(uint32_t w, uint32_t (&o)[4]) {
  asm("{ .reg .b8 b0, b1, b2, b3;\n"
      "mov.b32 {b0, b1, b2, b3}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n"
      "cvt.rn.f16x2.e2m1x2 %3, b3; }"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}
// four 8-bit integers -> two f16x2, exact: f16 numbers from 1024 to 2047 are 1024
// plus their low bits, so a byte v + 128 behind 0x64 reads as v + 1152
__device__ __forceinline__ void s8x4_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  asm("{ .reg .b32 c; mov.b32 c, 0x64806480; sub.rn.f16x2 %0, %2, c; sub.rn.f16x2 %1, %3, c; }"
      : "=r"(lo), "=r"(hi)
      : "r"(__byte_perm(u, 0x64646464u, 0x4140)), "r"(__byte_perm(u, 0x64646464u, 0x4342)));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace oes
