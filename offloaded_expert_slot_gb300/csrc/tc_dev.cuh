// Device helpers of the warp-specialised tcgen05 kernels: bounded waits that leave a
// CTA able to end, the uniform warp index, moves of registers between warps, and
// addresses and barriers of a cluster.
#pragma once

#include "common.cuh"

namespace oes {
namespace {

// Polls of the waits below; a test builds the products with few, so that they run out.
#ifndef OES_FP8_WAIT_POLLS
#define OES_FP8_WAIT_POLLS kWaitLimit
#endif

// The bounded waits of a CTA's warps, all lanes of a warp together.  One that
// gives up sets the status and the CTA's flag; from then on no wait lasts and
// nothing more is loaded, but every warp walks its loops to their end, so that
// no barrier between warps is left short, and drain() then waits for what is in
// flight.  That the first test stands alone, that no wait has an exit of its own
// and that the flag costs no register matters: with a result to test after each
// wait the FP8 product of 4096 x 8192 x 4096 took 131 us, with a flag in a register
// 119, like this 116.  LOOP_ASM: the loop in one asm block, 3 % better for the experts' kernels
// and 10 % worse for the dense one.
template <bool LOOP_ASM>
struct Waits {
  int32_t* status;
  volatile int* flag;
  __device__ __forceinline__ bool dead() const { return *flag != 0; }
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) {
    if (!mbar_try_wait(bar, parity)) slow(bar, parity);
  }
  __device__ __forceinline__ void slow(uint64_t* bar, uint32_t parity) {
    if (dead()) return;
    if (LOOP_ASM) {
      uint32_t ok;
      asm volatile(
          "{ .reg .pred p; .reg .u32 n; mov.u32 n, 0;\n"
          "W%=: mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
          "@p bra D%=;\n"
          "add.u32 n, n, 1;\n"
          "setp.lt.u32 p, n, %3;\n"
          "@p bra W%=;\n"
          "D%=: selp.u32 %0, 1, 0, p; }"
          : "=r"(ok)
          : "r"(smem_u32(bar)), "r"(parity), "n"(OES_FP8_WAIT_POLLS)
          : "memory");
      if (!ok) give_up();
    } else if (!mbar_wait(bar, parity, status, OES_FP8_WAIT_POLLS)) {
      *flag = 1;
    }
  }
  __device__ __forceinline__ void give_up() {
    set_status(status, OES_DEV_TIMEOUT);
    *flag = 1;
  }
  // arrivals and data come from other CTAs of the cluster
  __device__ __forceinline__ void cluster(uint64_t* bar, uint32_t parity) {
    for (uint32_t i = 0; i < OES_FP8_WAIT_POLLS; ++i) {
      uint32_t ok;
      asm volatile(
          "{ .reg .pred p; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2; selp.u32 "
          "%0, 1, 0, p; }"
          : "=r"(ok)
          : "r"(smem_u32(bar)), "r"(parity)
          : "memory");
      if (ok || dead()) return;
      if (i > 64) __nanosleep(32);
    }
    give_up();
  }
};

// 32 lanes x 32 columns
__device__ __forceinline__ void tmem_ld_32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, "
      "%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// The warp's index, in a form the compiler can see is the same for all lanes:
// what follows from it then needs no registers of each thread (the dense 256-wide
// tile's kernel stores 32 bytes a thread to local memory without, 16 with; with
// fp32 results 80 and none).
__device__ __forceinline__ int warp_index() { return __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0); }
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void named_bar(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// ----- clusters: a shared address of another CTA, and the barrier of all
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

}  // namespace
}  // namespace oes
