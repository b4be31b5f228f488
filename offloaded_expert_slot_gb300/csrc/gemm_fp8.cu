// Matrix products of e4m3 codes with block scales, on tcgen05 / TMEM / TMA:
// moe_fp8_gemm, and the grouped SwiGLU expert GEMM of moe_grouped_gemm_slots
// for the FP8 format.
//
//   out[t, n] = sum_b xs[t, b] ws[n / 128, b] sum_{k in b} x[t, k] w[n, k]
//
// over blocks b of 128 along K.  The scales are fp32 numbers, so they cannot
// go into the MMA: the tensor core sums the products of one block (four MMAs
// of K = 32, fp32 in tensor memory) and the epilogue warps scale each block's
// sums and add them to fp32 registers, block after block.  A block's sums go
// to one of several TMEM buffers, so that the MMAs of the next blocks run
// while the warps drain this one.
//
// h is rounded once, to its codes, and y, the down product's rows, once to bf16 as
// in the other formats: that is 2.4e-3 of relative error against 64 bits where
// fp32 rows would give 1.7e-3, and 0.34 GB less traffic at 4096 tokens x 10 x 2048.
//
// Two kernels share this; MODE 0 is the dense product, MODE 1 the experts'
// gate and up products with SwiGLU and h's codes, MODE 2 their down product.
//   token-major: 128 rows x 256 weight rows a tile (the experts' down product
//     128), for many rows.  The dense product is bound by the epilogue, which
//     has to scale and add each block's 128 x 256 sums while the tensor cores
//     make the next: 4096 x 8192 x 4096 takes 117 us, 2.35 PFLOP/s, with the
//     tensor pipe active for 52 % of them.  Tiles of 128 weight rows took 185
//     us there.  The experts' products are bound by the stream of weights: 4096
//     tokens x 10 of 512 experts (2048 x 768) read 1.7 GB for gate and up in
//     300 us, 5.7 TB/s, and move 1.0 GB for down in 156 us, 6.5 TB/s.
//   weight-major: 128 weight rows x 16 or 32 rows a tile, for few rows, bound
//     by the stream of weights: 32 tokens x 10 of the same experts read 763 MB
//     for gate and up in 120 us, 6.4 TB/s, and 382 MB for down in 68 us, 5.6
//     TB/s.  When the tiles do not fill the GPU, the CTAs of a cluster share a
//     tile's K range and add their sums over distributed shared memory in a
//     fixed order (1 x 1536 x 2048: 3.9 us).
#include <algorithm>

#include "common.cuh"
#include "fp8_dev.cuh"
#include "gemm_types.h"
#include "gemm_units.cuh"
#include "internal.h"

namespace oes {
namespace {

constexpr int kBlkK = 128;                 // codes (bytes) of K a pipeline stage holds
constexpr int kTileBytes = kTileM * kBlkK;  // 128 rows of one stage
constexpr int kEpiW0 = 4;                  // first epilogue warp

struct Fp8Maps {
  CUtensorMap w;  // weights [slots][rows][K], box 128 x 128
  CUtensorMap x;  // MODE 0: x [T][K]; MODE 2: h [cap][I]
};

struct Fp8Params {
  GemmParams g;      // grouped: routing tables and sizes; dense: status
  const uint8_t* x;  // MODE 1: codes of x, gathered
  const float* xs;   // scales of the rows of x (MODE 2: of h) [rows, nkb]
  const float* ws;   // dense: block scales of w; grouped: those of the pool's row 0
  int T, N, K, nkb;  // dense rows; weight rows (MODE 1: of gate, = I); K; blocks of K
  int mt, nt;        // dense: row tiles, weight tiles
  void* out;         // MODE 0 out, MODE 1 codes of h, MODE 2 y
  int64_t out_ld;
  int out_f32, vec;  // dense: type of out; its rows and their pieces are multiples of 16 bytes
  float* hs;         // MODE 1: scales of h
  int ks_log, ns;    // 2^ks_log CTAs share a tile's K range; pipeline stages
};

// A unit past the CTA's table, out of line: five roles look units up.  (The
// token-major kernel cannot call functions: it moves registers between warps.)
template <bool CG>
__device__ __noinline__ Unit unit_past_table(const GemmParams& g, int u, int nb) {
  return unit_info<CG>(g, u, nb);
}

// One unit of work: tile m of the weights against rows block b.
template <int MODE, bool TM>
__device__ __forceinline__ Unit unit_of(const Fp8Params& p, const UnitRec* tab, int idx, int u, int nb,
                                        int rows) {
  if (MODE == 0) {
    // row tiles fastest: the CTAs of a wave share a few weight tiles and
    // read x from L2
    Unit t;
    t.b = u % p.mt;
    t.m = u / p.mt;
    t.h = 0;
    t.slot = 0;
    t.nvalid = min(rows, p.T - t.b * rows);
    t.skip = false;
    return t;
  }
  if (idx >= kMaxUnitsPerCta)
    return TM ? unit_info<MODE == 2>(p.g, u, nb) : unit_past_table<MODE == 2>(p.g, u, nb);
  const UnitRec r = tab[idx];
  Unit t;
  t.b = r.b;
  t.m = r.m;
  t.h = 0;
  t.slot = r.slot;
  t.nvalid = r.nvalid;
  t.skip = t.slot < 0 || t.slot >= p.g.S || t.nvalid == 0;
  return t;
}

// Fills the CTA's unit table (grouped) and returns the number of units.
template <int MODE>
__device__ __forceinline__ int unit_table(const Fp8Params& p, UnitRec* utab, int* s_scan, int worker,
                                          int nworkers, int* nb_out) {
  if (MODE == 0) return p.mt * p.nt;
  const GemmParams& g = p.g;
  const int nb = ld_tab<MODE == 2>(g.n_post_pad) / g.BN;
  *nb_out = nb;
  if (g.filter) {
    const int dense = fill_filtered_units<MODE == 2>(g, nb, utab, s_scan, worker, nworkers);
    if (dense >= 0) return dense;
  }
  const int total = nb * g.n_mtiles;
  for (int i = threadIdx.x; i < kMaxUnitsPerCta; i += blockDim.x) {
    const int u = worker + i * nworkers;
    if (u >= total) break;
    const Unit t = unit_info<MODE == 2, true>(g, u, nb);
    utab[i] = UnitRec{t.b, t.m, t.slot, t.nvalid};
  }
  return total;
}

__device__ __forceinline__ const float* scales_of(const Fp8Params& p, int slot) {
  return reinterpret_cast<const float*>(reinterpret_cast<const uint8_t*>(p.ws) + (int64_t)slot * p.g.row_bytes);
}

// Polls of the waits below; a test builds this file with few, so that they run out.
#ifndef OES_FP8_WAIT_POLLS
#define OES_FP8_WAIT_POLLS kWaitLimit
#endif

// The bounded waits of a CTA's warps, all lanes of a warp together.  One that
// gives up sets the status and the CTA's flag; from then on no wait lasts and
// nothing more is loaded, but every warp walks its loops to their end, so that
// no barrier between warps is left short, and drain() then waits for what is in
// flight.  That the first test stands alone, that no wait has an exit of its own
// and that the flag costs no register matters: with a result to test after each
// wait 4096 x 8192 x 4096 took 131 us, with a flag in a register 119, like this
// 116.  LOOP_ASM: the loop in one asm block, 3 % better for the experts' kernels
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
// D[tmem] (+)= A[smem] * B[smem]^T, kind::f8f6f4 (e4m3 inputs, fp32 sums)
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, "
      "p; }" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// e4m3 x e4m3 -> fp32, both K-major, shape M x N
__device__ __forceinline__ uint32_t idesc_f8(uint32_t M, uint32_t N) {
  return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
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
// 16 bytes global -> shared, or 16 zero bytes
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst_smem, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst_smem), "l"(src), "r"(take ? 16 : 0)
               : "memory");
}
// 4 bytes global -> shared
__device__ __forceinline__ void cp_async4(uint32_t dst_smem, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst_smem), "l"(src) : "memory");
}
// Asynchronous copy of a row piece to global memory, by the thread that wrote
// it (16-byte aligned, a multiple of 16 bytes), and the thread's waits for its
// copies: until they have read shared memory, or until they are done.
__device__ __forceinline__ void bulk_store(void* dst, const void* src, int bytes) {
  fence_proxy_async_smem();
  asm volatile(
      "cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n"
      "cp.async.bulk.commit_group;" ::"l"(dst),
      "r"(smem_u32(src)), "r"(bytes)
      : "memory");
}
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void named_bar(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ----- clusters: a shared address of another CTA, and its barriers
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
// Into another CTA's shared memory, the bytes counted by a barrier there: whoever
// waits for that barrier sees them.  With plain stores, a fence and a releasing
// arrival 1 x 1536 x 2048 took 5.4 us, like this 3.9.
__device__ __forceinline__ void st_async(uint32_t addr, float v, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(addr),
               "r"(__float_as_uint(v)), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Once every role of a CTA in which a wait gave up has ended, by one thread: no
// copy and no MMA of the CTA outlives its shared memory and TMEM.  fills[r] is
// the number of stages that producer r filled (0 the weights; then the rows, or in
// MODE 1 the four gather warps).  A fill's phase ends when all its arrivals and
// bytes are in; what a producer that stopped before it owes is arrived here, for
// the ring's last ns fills (the stages of earlier ones were released, so their
// phases have ended).  mma_done ends with the issuer's last MMA.  Called by the
// warp that frees the TMEM: by all warps' common tail it took registers from the
// loops (4096 tokens x 10: 512 us, like this 503).
template <int MODE>
__device__ __forceinline__ void drain(uint64_t* full, int ns, const volatile int* fills, uint64_t* mma_done,
                                      int32_t* status) {
  constexpr int kProducers = MODE == 1 ? 5 : 2;
  int most = 0;
#pragma unroll 1
  for (int r = 0; r < kProducers; ++r) most = max(most, fills[r]);
#pragma unroll 1
  for (int i = max(0, most - ns); i < most; ++i) {
    uint64_t* bar = &full[i % ns];
#pragma unroll 1
    for (int r = 0; r < kProducers; ++r) {
      if (fills[r] > i) continue;
#pragma unroll 1
      for (int n = MODE == 1 && r > 0 ? 32 : 1; n > 0; --n) mbar_arrive(bar);
    }
    mbar_wait(bar, (i / ns) & 1, status);
  }
  mbar_wait(mma_done, 0, status);
}

// ============================================================ token-major
// TN weight rows a tile (MODE 1: 128 gate + 128 up).  TMEM holds 512 / TN
// blocks' sums.
__host__ __device__ constexpr int tm_stage(int TN) { return (TN + kTileM) * kBlkK; }
constexpr int kTmEpi = 8;     // epilogue warps: two a TMEM lane quarter, 128 columns each
constexpr int kTmGatherW0 = kEpiW0 + kTmEpi;
// Scales reach the epilogue through shared memory, fetched ahead by warp 2
// like the operands: read from global memory by the epilogue itself, one
// block ahead, their latency set the pace (4096 x 8192 x 4096: 160 us, then 144).
// A slot holds 8 blocks of K: [block][row] of x, [2][block] of the weights.
constexpr int kTmScK = 8;
constexpr int kTmScFloats = kTmScK * (kTileM + 2);
constexpr int kScSlots = 2;
// Results leave through shared memory, since 16-byte stores to 32 different rows
// at a time cost 4 us a tile.  The dense and the down product turn pieces of 64
// bytes of 32 rows around in 2 KB a warp and store them in whole sectors.  h's
// codes are copied out asynchronously, a thread its row's 64 bytes (rows 80
// bytes apart, so that eight lanes never meet in a bank).
__host__ __device__ constexpr int stg_row(int mode) {
  return mode == 1 ? 64 + 16 : 64;
}
__host__ __device__ constexpr int tm_threads(int mode) { return mode == 1 ? 512 : 384; }

// Registers: the launch gives every thread 65536 / threads; the epilogue
// warps (128 sums each) take what the other warpgroups give back.
// MODE 1: 512 x 128 = 128 (56 + 2 x 200 + 56).  Else 384 x 168 = 128 (72 + 2 x
// 216), with fp32 results 128 (56 + 2 x 224): 4096 x 4096 x 4096 takes 76 us, 96
// with the first split.
template <int MODE, typename OT, int TN>
__global__ void __launch_bounds__(tm_threads(MODE), 1)
    fp8_tm_kernel(const __grid_constant__ Fp8Maps maps, const __grid_constant__ Fp8Params p) {
  constexpr int kStage = tm_stage(TN);
  constexpr int kBufs = 512 / TN;
  constexpr int kCols = TN / 2;  // columns of an epilogue warp
  constexpr int kStgRow = stg_row(MODE);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stages =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(stages + p.ns * kStage);
  uint64_t* empty = full + p.ns;
  uint64_t* tfull = empty + p.ns;
  uint64_t* tempty = tfull + kBufs;
  uint64_t* sfull = tempty + kBufs;
  uint64_t* sempty = sfull + kScSlots;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sempty + kScSlots);
  UnitRec* utab = reinterpret_cast<UnitRec*>(tmem_holder + 4);
  uint8_t* stg_all = reinterpret_cast<uint8_t*>(utab + (MODE == 0 ? 0 : kMaxUnitsPerCta));
  float* sc_tab = reinterpret_cast<float*>(stg_all + kTmEpi * 32 * kStgRow);
  __shared__ int s_scan[33];
  __shared__ float s_amax[2][2][kTileM];
  const int warp = warp_index(), lane = threadIdx.x & 31;
  __shared__ int s_dead, s_fills[5];  // see drain()
  __shared__ uint64_t s_mma_done;
  Waits<MODE != 0> wait{p.g.status, &s_dead};
  if (threadIdx.x == 0) {
    s_dead = 0;
    for (int r = 0; r < 5; ++r) s_fills[r] = 0;
    mbar_init(&s_mma_done, 1);
    for (int s = 0; s < p.ns; ++s) {
      // the weights' TMA, and the rows' TMA or gather threads
      mbar_init(&full[s], 1 + (MODE == 1 ? 128 : 1));
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < kBufs; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], kTmEpi);
    }
    for (int a = 0; a < kScSlots; ++a) {
      mbar_init(&sfull[a], 32);
      mbar_init(&sempty[a], kTmEpi);
    }
    fence_mbar_init();
    tma_prefetch_desc(&maps.w);
    if (MODE != 1) tma_prefetch_desc(&maps.x);
  }
  // The gate and up product releases the down product once its units are known;
  // a CTA of that starts where one of this ends, and waits for h alone (see the
  // weight-major kernel).  600 tokens x 10 routes took 159 us so, 162 where it
  // waits first; 4096 tokens 498 and 502.
  if (MODE != 2) pdl_wait();
  if (MODE != 0 && p.g.filter && p.g.gcount && ld_tab<MODE == 2>(p.g.gcount + p.g.filter) == 0) return;
  int nb = 0;
  const int total = unit_table<MODE>(p, utab, s_scan, blockIdx.x, gridDim.x, &nb);
  __syncthreads();
  if ((int)blockIdx.x >= total) return;
  if (MODE == 1) pdl_trigger();
  if (warp == 2) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  if (warp < kEpiW0) {
    if (TN == 256) regs_dec<MODE == 1 || sizeof(OT) == 4 ? 56 : 72>();
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------- weight producer
      int s = 0, ph = 0;  // the next stage; times around the ring
      for (int u = blockIdx.x, ui = 0; u < total; u += gridDim.x, ++ui) {
        const Unit t = unit_of<MODE, true>(p, utab, ui, u, nb, kTileM);
        if (t.skip) continue;
        const int ra = t.m * (MODE == 1 ? kTileM : TN);
        const int rb = MODE == 1 ? p.N + ra : ra + kTileM;
#pragma unroll 1
        for (int kb = 0; kb < p.nkb; ++kb) {
          wait(&empty[s], ~ph & 1);
          if (wait.dead()) break;
          uint8_t* W = stages + s * kStage;
          mbar_arrive_expect_tx(&full[s], TN * kBlkK);
          tma_load_3d(W, &maps.w, &full[s], kb * kBlkK, ra, t.slot);
          if (TN == 256) tma_load_3d(W + kTileBytes, &maps.w, &full[s], kb * kBlkK, rb, t.slot);
          if (++s == p.ns) { s = 0; ++ph; }
        }
      }
      s_fills[0] = ph * p.ns + s;
    } else if (warp == 1) {
      // -------------------------------------------------------- MMA issuer
      // The whole warp walks the loop and one elected lane issues, so that the
      // descriptors stay in uniform registers: issued from a one-lane branch,
      // each hand-off took 0.09 us longer.
      int s = 0, ph = 0;
      uint32_t it = 0;
      const uint32_t idesc = idesc_f8(kTileM, TN);
      const uint64_t desc0 = smem_desc_sw128(smem_u32(stages));
      const bool leader = elect_one();
      for (int u = blockIdx.x, ui = 0; u < total; u += gridDim.x, ++ui) {
        const Unit t = unit_of<MODE, true>(p, utab, ui, u, nb, kTileM);
        if (t.skip) continue;
#pragma unroll 1
        for (int kb = 0; kb < p.nkb; ++kb, ++it) {
          const uint32_t a = it % kBufs;
          wait(&full[s], ph);
          wait(&tempty[a], ((it / kBufs) & 1) ^ 1);
          tc_fence_after();
          if (MODE == 1) fence_proxy_async_smem();  // cp.async-written rows -> tensor core
          if (leader) {
            const uint64_t wd = desc0 + (uint32_t)(s * (kStage >> 4)), xd = wd + (TN * kBlkK >> 4);
#pragma unroll
            for (int kk = 0; kk < kBlkK / 32; ++kk)
              tc_mma_f8(tmem_base + a * TN, xd + 2 * kk, wd + 2 * kk, idesc, kk ? 1u : 0u);
            tc_commit(&empty[s]);
            tc_commit(&tfull[a]);
          }
          __syncwarp();
          if (++s == p.ns) { s = 0; ph ^= 1; }
        }
      }
      if (leader) tc_commit(&s_mma_done);
    } else if (warp == 2) {
      // ---------------------------------------------------- scale producer
      // lane l: rows l + 32 i and, of the weights' 2 x 8 scales, one
      const int nwb = (p.N + 127) / 128;  // blocks of weight rows
      uint32_t n = 0;
      if (MODE == 2) pdl_wait();  // h's scales
      for (int u = blockIdx.x, ui = 0; u < total; u += gridDim.x, ++ui) {
        const Unit t = unit_of<MODE, true>(p, utab, ui, u, nb, kTileM);
        if (t.skip) continue;
        const float* xr[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = lane + 32 * i;
          int64_t r = 0;  // rows past the block's last: any scale does
          if (row < t.nvalid) {
            const int64_t at = (int64_t)t.b * kTileM + row;
            r = MODE == 1 ? p.g.sorted_ids[at] / p.g.k : at;
          }
          xr[i] = p.xs + r * p.nkb;
        }
        // MODE 1: the gate's and the up's row of blocks; else the two halves'
        const int h = (lane >> 3) & 1, wb = MODE == 1 ? t.m + h * nwb : TN == 256 ? 2 * t.m + h : t.m;
        const float* wr = (MODE == 0 ? p.ws : scales_of(p, t.slot)) +
                          (int64_t)(MODE == 1 || wb < nwb ? wb : wb - 1) * p.nkb;
        for (int k0 = 0; k0 < p.nkb; k0 += kTmScK, ++n) {
          const int slot = n % kScSlots;
          wait(&sempty[slot], ((n / kScSlots) & 1) ^ 1);
          if (__any_sync(0xffffffffu, wait.dead())) break;
          float* tab = sc_tab + slot * kTmScFloats;
          const int kn = min(kTmScK, p.nkb - k0);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            for (int k = 0; k < kn; ++k)
              cp_async4(smem_u32(tab + k * kTileM + lane + 32 * i), xr[i] + k0 + k);
          if (lane < 16 && (lane & 7) < kn)
            cp_async4(smem_u32(tab + kTmScK * kTileM + lane), wr + k0 + (lane & 7));
          cp_async_mbar_arrive(&sfull[slot]);
        }
      }
      cp_async_wait_all();
    } else if (MODE != 1 && warp == 3 && lane == 0) {
      // ------------------------------------------------------ rows producer
      int s = 0, ph = 0;  // the next stage; times around the ring
      if (MODE == 2) pdl_wait();  // h is the kernel before's output
      for (int u = blockIdx.x, ui = 0; u < total; u += gridDim.x, ++ui) {
        const Unit t = unit_of<MODE, true>(p, utab, ui, u, nb, kTileM);
        if (t.skip) continue;
#pragma unroll 1
        for (int kb = 0; kb < p.nkb; ++kb) {
          wait(&empty[s], ~ph & 1);
          if (wait.dead()) break;
          mbar_arrive_expect_tx(&full[s], kTileBytes);
          tma_load_2d(stages + s * kStage + TN * kBlkK, &maps.x, &full[s], kb * kBlkK, t.b * kTileM);
          if (++s == p.ns) { s = 0; ++ph; }
        }
      }
      s_fills[1] = ph * p.ns + s;
    }
  } else if (warp < kTmGatherW0) {
    if (TN == 256) regs_inc<MODE == 1 ? 200 : sizeof(OT) == 4 ? 224 : 216>();
    // ---------------------------------------------------------- epilogue
    const int q = warp & 3, half = (warp - kEpiW0) >> 2;
    const int row = q * 32 + lane;  // TMEM lane = row of the tile
    const int nwb = (p.N + 127) / 128;  // blocks of weight rows
    // this warp's staged rows, and this thread's
    uint8_t* const stg = stg_all + (warp - kEpiW0) * 32 * kStgRow;
    uint8_t* const mine = stg + lane * kStgRow;
    uint32_t it = 0, sn = 0;
    int par = 0;
    for (int u = blockIdx.x, ui = 0; u < total; u += gridDim.x, ++ui) {
      const Unit t = unit_of<MODE, true>(p, utab, ui, u, nb, kTileM);
      const bool live = row < t.nvalid;
      const int col0 = t.m * TN + half * kCols;  // MODE 0, 2: first column of this warp
      int r = 0;                                    // row of out (MODE 2: the route)
      if (MODE == 2 && live) r = ld_tab<true>(p.g.sorted_ids + (int64_t)t.b * p.g.BN + row);
      if (t.skip) {
        if (MODE == 2 && live && t.slot != kFiltered) {
          // an expert without a slot: its routes get zeros (and a status bit)
          uint16_t* y = static_cast<uint16_t*>(p.out) + (int64_t)r * p.out_ld;
          for (int c = col0; c < min(col0 + kCols, p.N); c += 8)
            *reinterpret_cast<uint4*>(y + c) = make_uint4(0, 0, 0, 0);
          if (row == 0) set_status(p.g.status, OES_DEV_BAD_ID);
        }
        continue;
      }
      const bool on = q * 32 < t.nvalid && (MODE == 1 ? t.m * kTileM + half * 64 : col0) < p.N;
      float acc[kCols];
#pragma unroll
      for (int j = 0; j < kCols; ++j) acc[j] = 0.0f;
      // Columns of this warp's piece c of 32: MODE 1 takes 64 gate columns and
      // the same 64 up columns, so that a thread has both factors of its h.
      constexpr int kPieces = kCols / 32;
      auto piece = [&](int c) {
        return MODE == 1 ? (c >> 1) * kTileM + half * 64 + (c & 1) * 32 : half * kCols + c * 32;
      };
#pragma unroll 1
      for (int k0 = 0; k0 < p.nkb; k0 += kTmScK, ++sn) {
        const int slot = sn % kScSlots;
        wait(&sfull[slot], (sn / kScSlots) & 1);
        const float* xt = sc_tab + slot * kTmScFloats + row;
        const float* wt = sc_tab + slot * kTmScFloats + kTmScK * kTileM + (MODE == 1 || TN == 128 ? 0 : half * kTmScK);
        float s0 = xt[0] * wt[0], s1 = MODE == 1 ? xt[0] * wt[kTmScK] : s0;
        const int kn = min(kTmScK, p.nkb - k0);
#pragma unroll 1
        for (int ki = 0; ki < kn; ++ki, ++it) {
          const uint32_t a = it % kBufs;
          wait(&tfull[a], (it / kBufs) & 1);
          tc_fence_after();
          // the next block's scales come in while this one's sums do
          xt += kTileM;
          ++wt;
          const bool more = ki + 1 < kn;
          const float xn = more ? xt[0] : 0.0f, w0 = more ? wt[0] : 0.0f;
          const float w1 = MODE == 1 && more ? wt[kTmScK] : 0.0f;
          if (on) {
            // the loads of one piece run under the FMAs of the one before
            const uint32_t tl = tmem_base + ((uint32_t)(q * 32) << 16) + a * TN;
            uint32_t d[2][32];
            tmem_ld_32(tl + piece(0), d[0]);
#pragma unroll
            for (int c = 0; c < kPieces; ++c) {
              tc_wait_ld();
              if (c + 1 < kPieces) {
                tmem_ld_32(tl + piece(c + 1), d[(c + 1) & 1]);
              } else {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&tempty[a]);
              }
#pragma unroll
              for (int j = 0; j < 32; ++j)
                acc[c * 32 + j] = fmaf(__uint_as_float(d[c & 1][j]), c >= kPieces / 2 ? s1 : s0, acc[c * 32 + j]);
            }
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[a]);
          }
          s0 = xn * w0;
          s1 = MODE == 1 ? xn * w1 : s0;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sempty[slot]);
      }
      if (MODE == 1) {
        if (q * 32 >= t.nvalid) continue;  // both warps of the quarter
        // h, the amax of its 128 columns with the other half's warp, codes
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < 64; ++j) {
          acc[j] = silu_f32(acc[j]) * acc[kCols / 2 + j];
          m = fmaxf(m, fabsf(acc[j]));
        }
        if (!on) m = 0.0f;
        s_amax[par][half][row] = m;
        named_bar(1 + q, 64);
        const QuantScale qs = quant_scale(fmaxf(m, s_amax[par][half ^ 1][row]));
        par ^= 1;
        if (live) {
          const int64_t hr = (int64_t)t.b * p.g.BN + row;
          if (on) {
            bulk_wait_read();  // the tile before has left this row
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float* v = acc + c * 16 + 4 * i;
                w[i] = quant4(v[0], v[1], v[2], v[3], qs);
              }
              *reinterpret_cast<uint4*>(mine + c * 16) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            bulk_store(static_cast<uint8_t*>(p.out) + hr * p.out_ld + t.m * kTileM + half * 64, mine, 64);
          }
          if (half == 0) p.hs[hr * nwb + t.m] = qs.s;
        }
      } else if (on) {
        constexpr int kPer = 64 / (int)sizeof(OT);  // columns of a piece
        constexpr int kVec = 16 / (int)sizeof(OT);
        if (MODE == 0) r = t.b * kTileM + row;
#pragma unroll
        for (int pc = 0; pc < kCols / kPer; ++pc) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float* v = acc + pc * kPer + c * kVec;
              if constexpr (sizeof(OT) == 2) w[i] = f32x2_bf16x2(v[2 * i], v[2 * i + 1]);
              else w[i] = __float_as_uint(v[i]);
            }
            *reinterpret_cast<uint4*>(stg + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int rr = 8 * i + (lane >> 2), c = lane & 3;
            const int ro = __shfl_sync(0xffffffffu, r, rr);
            const int col = col0 + pc * kPer + c * kVec;
            const uint8_t* from = stg + rr * 64 + ((c ^ ((rr >> 1) & 3)) << 4);
            if (q * 32 + rr < t.nvalid && col < p.N) {
              OT* o = static_cast<OT*>(p.out) + (int64_t)ro * p.out_ld + col;
              if (MODE == 2 || (p.vec && col + kVec <= p.N)) {
                *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(from);
              } else {
#pragma unroll 1
                for (int e = 0; e < min(kVec, p.N - col); ++e) o[e] = reinterpret_cast<const OT*>(from)[e];
              }
            }
          }
          __syncwarp();
        }
      }
    }
    if (MODE == 1) bulk_wait_all();  // the copies out of this CTA's shared memory
  } else if (MODE == 1) {
    regs_dec<56>();
    // ------------------------------------------------------- token gather
    // thread g copies 16-byte chunk g % 8 of rows g / 8 + 16 j; its copies
    // arrive on the stage's barrier when they complete.  Bytes past H (its
    // last block may be half of one) are zeros: a weight's zero there would
    // not silence a NaN code.
    const int g = threadIdx.x - kTmGatherW0 * 32;
    const int c = g & 7, r0 = g >> 3;
    int s = 0, ph = 0;  // the next stage; times around the ring
    for (int u = blockIdx.x, ui = 0; u < total; u += gridDim.x, ++ui) {
      const Unit t = unit_of<MODE, true>(p, utab, ui, u, nb, kTileM);
      if (t.skip) continue;
      const int n16 = round16(t.nvalid);
      const uint8_t* src[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int n = r0 + 16 * j;
        const int tk = n < t.nvalid ? p.g.sorted_ids[(int64_t)t.b * p.g.BN + n] / p.g.k : 0;
        src[j] = p.x + (int64_t)tk * p.K + c * 16;
      }
#pragma unroll 1
      for (int kb = 0; kb < p.nkb; ++kb) {
        wait(&empty[s], ~ph & 1);
        if (__any_sync(0xffffffffu, wait.dead())) break;
        const uint32_t X = smem_u32(stages + s * kStage + TN * kBlkK);
        const bool in = kb * kBlkK + c * 16 < p.K;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int n = r0 + 16 * j;
          if (n < n16) cp_async16_or_zero(X + n * kBlkK + ((c ^ (n & 7)) << 4), in ? src[j] + kb * kBlkK : src[j], in);
        }
        cp_async_mbar_arrive(&full[s]);
        if (++s == p.ns) { s = 0; ++ph; }
      }
    }
    cp_async_wait_all();
    if (lane == 0) s_fills[1 + warp - kTmGatherW0] = ph * p.ns + s;
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    if (wait.dead()) {
      if (lane == 0) drain<MODE>(full, p.ns, s_fills, &s_mma_done, p.g.status);
      __syncwarp();
    }
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// =========================================================== weight-major
// BN rows a tile (16; the dense product 32 too).  Warps: 0 weights, 1 MMA,
// 2 TMEM, 3 rows (TMA), 4-7 epilogue, 8-11 token gather (MODE 1).
constexpr int kWmAcc = 4;  // TMEM buffers
// A slot of scales (see above) holds 32 blocks of K: [block][BN] of the rows,
// [kA][block] of the weights.
constexpr int kWmScK = 32;
__host__ __device__ constexpr int wm_sc_floats(int mode, int BN) { return kWmScK * (BN + (mode == 1 ? 2 : 1)); }
__host__ __device__ constexpr int wm_threads(int mode) { return mode == 1 ? 384 : 256; }
__host__ __device__ constexpr int wm_stage(int mode, int BN) {
  return (mode == 1 ? 2 : 1) * kTileBytes + BN * kBlkK;
}

template <int MODE, int BN>
__global__ void __launch_bounds__(wm_threads(MODE), 1)
    fp8_wm_kernel(const __grid_constant__ Fp8Maps maps, const __grid_constant__ Fp8Params p) {
  constexpr int kA = MODE == 1 ? 2 : 1;  // weight tiles a stage (gate and up)
  constexpr int kStage = wm_stage(MODE, BN);
  constexpr uint32_t kCols = kWmAcc * kA * BN;  // TMEM columns: 64 or 128
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stages =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* red = reinterpret_cast<float*>(stages + p.ns * kStage);  // [kA][ks][BN / ks][128]
  uint64_t* full = reinterpret_cast<uint64_t*>(red + kA * BN * kTileM);
  uint64_t* empty = full + p.ns;
  uint64_t* tfull = empty + p.ns;
  uint64_t* tempty = tfull + kWmAcc;
  uint64_t* rfull = tempty + kWmAcc;  // [4]: a warp's sums of every CTA of the cluster are in
  uint64_t* sfull = rfull + 4;
  uint64_t* sempty = sfull + kScSlots;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sempty + kScSlots);
  UnitRec* utab = reinterpret_cast<UnitRec*>(tmem_holder + 4);
  float* sc_tab = reinterpret_cast<float*>(utab + kMaxUnitsPerCta);
  constexpr int kScFloats = wm_sc_floats(MODE, BN);
  __shared__ int s_scan[33];
  __shared__ float s_amax[2][4][BN];
  const int warp = warp_index(), lane = threadIdx.x & 31;
  __shared__ int s_dead, s_fills[5];  // see drain()
  __shared__ uint64_t s_mma_done;
  Waits<true> wait{p.g.status, &s_dead};
  // the CTAs of a cluster have neighbouring block indices
  const int ks = 1 << p.ks_log, rank = (int)blockIdx.x & (ks - 1);
  const int worker = (int)blockIdx.x >> p.ks_log, nworkers = (int)gridDim.x >> p.ks_log;
  const int k_lo = (rank * p.nkb) >> p.ks_log, k_hi = ((rank + 1) * p.nkb) >> p.ks_log;
  if (threadIdx.x == 0) {
    s_dead = 0;
    for (int r = 0; r < 5; ++r) s_fills[r] = 0;
    mbar_init(&s_mma_done, 1);
    for (int s = 0; s < p.ns; ++s) {
      mbar_init(&full[s], 1 + (MODE == 1 ? 128 : 1));
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < kWmAcc; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 4);
    }
    for (int w = 0; w < 4; ++w) mbar_init(&rfull[w], 1);
    for (int a = 0; a < kScSlots; ++a) {
      mbar_init(&sfull[a], 32);
      mbar_init(&sempty[a], 4);
    }
    fence_mbar_init();
    tma_prefetch_desc(&maps.w);
    if (MODE != 1) tma_prefetch_desc(&maps.x);
  }
  // The down product is launched while the gate and up product runs (which
  // releases it after its set-up): all it reads but h was complete before
  // that kernel passed this wait, so it builds its unit table and streams its
  // first weights now, and only what reads h waits (below).  Tables it reads
  // without waiting are read through L2.  32 tokens x 10 of 512 experts: 187 us,
  // 193 with the release left to the end where a CTA has more than two units; 64
  // x 8 of 64: 75 and 80.
  if (MODE != 2) pdl_wait();
  if (MODE != 0 && p.g.filter && p.g.gcount && ld_tab<MODE == 2>(p.g.gcount + p.g.filter) == 0) return;
  int nb = 0;
  const int total = unit_table<MODE>(p, utab, s_scan, worker, nworkers, &nb);
  __syncthreads();
  if (worker >= total) return;  // the whole cluster
  if (warp == 2) {
    tmem_alloc(tmem_holder, kCols);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  if (ks > 1) cluster_barrier();  // every CTA's barriers are initialised
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  if (MODE == 1) pdl_trigger();
  bool awaited = false;  // an epilogue warp: the cluster's CTAs send it sums

  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------------- weight producer
      int s = 0, ph = 0;  // the next stage; times around the ring
      for (int u = worker, ui = 0; u < total; u += nworkers, ++ui) {
        const Unit t = unit_of<MODE, false>(p, utab, ui, u, nb, BN);
        if (t.skip) continue;
#pragma unroll 1
        for (int kb = k_lo; kb < k_hi; ++kb) {
          wait(&empty[s], ~ph & 1);
          if (wait.dead()) break;
          uint8_t* W = stages + s * kStage;
          mbar_arrive_expect_tx(&full[s], kA * kTileBytes);
          tma_load_3d(W, &maps.w, &full[s], kb * kBlkK, t.m * kTileM, t.slot);
          if (MODE == 1)
            tma_load_3d(W + kTileBytes, &maps.w, &full[s], kb * kBlkK, p.N + t.m * kTileM, t.slot);
          if (++s == p.ns) { s = 0; ++ph; }
        }
      }
      s_fills[0] = ph * p.ns + s;
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    int s = 0, ph = 0;
    uint32_t it = 0;
    const uint64_t desc0 = smem_desc_sw128(smem_u32(stages));
    const bool leader = elect_one();
    for (int u = worker, ui = 0; u < total; u += nworkers, ++ui) {
      const Unit t = unit_of<MODE, false>(p, utab, ui, u, nb, BN);
      if (t.skip) continue;
      const uint32_t idesc = idesc_f8(kTileM, round16(t.nvalid));
#pragma unroll 1
      for (int kb = k_lo; kb < k_hi; ++kb, ++it) {
        const uint32_t a = it % kWmAcc;
        wait(&full[s], ph);
        wait(&tempty[a], ((it / kWmAcc) & 1) ^ 1);
        tc_fence_after();
        if (MODE == 1) fence_proxy_async_smem();
        if (leader) {
          const uint64_t wd = desc0 + (uint32_t)(s * (kStage >> 4)), xd = wd + (kA * kTileBytes >> 4);
          const uint32_t d = tmem_base + a * kA * BN;
#pragma unroll
          for (int kk = 0; kk < kBlkK / 32; ++kk) {
            tc_mma_f8(d, wd + 2 * kk, xd + 2 * kk, idesc, kk ? 1u : 0u);
            if (MODE == 1)
              tc_mma_f8(d + BN, wd + (kTileBytes >> 4) + 2 * kk, xd + 2 * kk, idesc, kk ? 1u : 0u);
          }
          tc_commit(&empty[s]);
          tc_commit(&tfull[a]);
        }
        __syncwarp();
        if (++s == p.ns) { s = 0; ph ^= 1; }
      }
    }
    if (leader) tc_commit(&s_mma_done);
  } else if (warp == 2) {
    // ------------------------------------------------------ scale producer
    if (MODE == 2) pdl_wait();  // h's scales
    const int nwb = (p.N + 127) / 128;
    uint32_t i = 0;
    for (int u = worker, ui = 0; u < total; u += nworkers, ++ui) {
      const Unit t = unit_of<MODE, false>(p, utab, ui, u, nb, BN);
      if (t.skip) continue;
      int tk = 0;  // MODE 1: the rows' tokens, one a lane
      if (MODE == 1 && lane < t.nvalid) tk = p.g.sorted_ids[(int64_t)t.b * p.g.BN + lane] / p.g.k;
      const float* w = (MODE == 0 ? p.ws : scales_of(p, t.slot)) + (int64_t)t.m * p.nkb;
      for (int k0 = k_lo; k0 < k_hi; k0 += kWmScK, ++i) {
        const int slot = i % kScSlots, k = k0 + lane;
        wait(&sempty[slot], ((i / kScSlots) & 1) ^ 1);
        if (__any_sync(0xffffffffu, wait.dead())) break;
        float* tab = sc_tab + slot * kScFloats;
        for (int n = 0; n < t.nvalid; ++n) {
          const int r = MODE == 1 ? __shfl_sync(0xffffffffu, tk, n & 31) : t.b * BN + n;
          if (k < k_hi) cp_async4(smem_u32(tab + lane * BN + n), p.xs + (int64_t)r * p.nkb + k);
        }
        if (k < k_hi) {
          cp_async4(smem_u32(tab + kWmScK * BN + lane), w + k);
          if (MODE == 1) cp_async4(smem_u32(tab + kWmScK * (BN + 1) + lane), w + (int64_t)nwb * p.nkb + k);
        }
        cp_async_mbar_arrive(&sfull[slot]);
      }
    }
    cp_async_wait_all();
  } else if (warp == 3) {
    if (MODE != 1 && lane == 0) {
      // ------------------------------------------------------ rows producer
      if (MODE == 2) pdl_wait();  // h is the kernel before's output
      int s = 0, ph = 0;  // the next stage; times around the ring
      for (int u = worker, ui = 0; u < total; u += nworkers, ++ui) {
        const Unit t = unit_of<MODE, false>(p, utab, ui, u, nb, BN);
        if (t.skip) continue;
#pragma unroll 1
        for (int kb = k_lo; kb < k_hi; ++kb) {
          wait(&empty[s], ~ph & 1);
          if (wait.dead()) break;
          mbar_arrive_expect_tx(&full[s], BN * kBlkK);
          tma_load_2d(stages + s * kStage + kA * kTileBytes, &maps.x, &full[s], kb * kBlkK, t.b * BN);
          if (++s == p.ns) { s = 0; ++ph; }
        }
      }
      s_fills[1] = ph * p.ns + s;
    }
  } else if (warp >= kEpiW0 && warp < kEpiW0 + 4) {
    // ---------------------------------------------------------- epilogue
    const int q = warp & 3;
    const int row = q * 32 + lane;  // TMEM lane = weight row of the tile
    const int nwb = (p.N + 127) / 128;
    // log2 of the columns this CTA finishes, from rank * own
    const int own_log = (BN == 16 ? 4 : 5) - p.ks_log, own = 1 << own_log;
    uint32_t it = 0, un = 0, sn = 0;
    for (int u = worker, ui = 0; u < total; u += nworkers, ++ui) {
      const Unit t = unit_of<MODE, false>(p, utab, ui, u, nb, BN);
      const int wrow = t.m * kTileM + row;
      if (t.skip) {
        if (MODE == 2 && t.nvalid > 0 && t.slot != kFiltered && rank == 0) {
          // an expert without a slot: its routes get zeros (and a status bit)
          if (wrow < p.N)
            for (int n = 0; n < t.nvalid; ++n)
              static_cast<uint16_t*>(p.out)[(int64_t)ld_tab<MODE == 2>(p.g.sorted_ids + (int64_t)t.b * p.g.BN + n) * p.out_ld + wrow] = 0;
          if (row == 0) set_status(p.g.status, OES_DEV_BAD_ID);
        }
        continue;
      }
      // MODE 2: the block's routes, one a lane
      int sid = 0;
      if (MODE == 2 && lane < t.nvalid) sid = ld_tab<true>(p.g.sorted_ids + (int64_t)t.b * p.g.BN + lane);
      float acc[kA][BN];
#pragma unroll
      for (int i = 0; i < kA; ++i)
#pragma unroll
        for (int n = 0; n < BN; ++n) acc[i][n] = 0.0f;
#pragma unroll 1
      for (int kb = k_lo; kb < k_hi; ++kb, ++it) {
        const uint32_t a = it % kWmAcc;
        const int slot = sn % kScSlots, ki = (kb - k_lo) % kWmScK;
        if (ki == 0) {
          wait(&sfull[slot], (sn / kScSlots) & 1);
        }
        wait(&tfull[a], (it / kWmAcc) & 1);
        tc_fence_after();
        const float* tab = sc_tab + slot * kScFloats;
        const uint32_t tl = tmem_base + ((uint32_t)(q * 32) << 16) + a * kA * BN;
#pragma unroll
        for (int c = 0; c < BN; c += 16) {
          if (c >= t.nvalid) continue;
          uint32_t d[kA][16];
#pragma unroll
          for (int i = 0; i < kA; ++i) tmem_ld_16(tl + i * BN + c, d[i]);
          float x[16];
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const float4 v = *reinterpret_cast<const float4*>(tab + ki * BN + c + j);
            x[j] = v.x; x[j + 1] = v.y; x[j + 2] = v.z; x[j + 3] = v.w;
          }
          tc_wait_ld();
#pragma unroll
          for (int i = 0; i < kA; ++i) {
            const float w = tab[kWmScK * (BN + i) + ki];
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[i][c + j] = fmaf(__uint_as_float(d[i][j]), x[j] * w, acc[i][c + j]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[a]);
        if (ki == kWmScK - 1 || kb == k_hi - 1) {
          if (lane == 0) mbar_arrive(&sempty[slot]);
          ++sn;
        }
      }
      // The sums go through shared memory, so that what follows is a loop
      // over columns: unrolled over registers it was 250 KB of code, and
      // fetching it took longer than the product.  Each CTA of a cluster
      // finishes `own` columns: it sends the others theirs and adds up its
      // own in rank order.
      const int n0 = rank << own_log, mine = min(own, t.nvalid - n0);
      const uint32_t base = smem_u32(red) + row * 4;
      if (ks > 1) {
        awaited = mine > 0;
        if (lane == 0 && awaited) mbar_arrive_expect_tx(&rfull[q], ks * kA * mine * 32 * 4);
#pragma unroll
        for (int n = 0; n < BN; ++n) {
          if (n >= t.nvalid) continue;
          const int d = n >> own_log, j = n & (own - 1);
          const uint32_t to = map_rank(base + (((rank << own_log) + j) * kTileM) * 4, d);
          const uint32_t bar = map_rank(smem_u32(&rfull[q]), d);
#pragma unroll
          for (int i = 0; i < kA; ++i) st_async(to + i * (BN * kTileM * 4), acc[i][n], bar);
        }
        if (awaited) wait.cluster(&rfull[q], 0);  // a cluster has one unit at most
      } else {
#pragma unroll
        for (int n = 0; n < BN; ++n) {
          if (n >= t.nvalid) continue;
#pragma unroll
          for (int i = 0; i < kA; ++i) red[(i * BN + n) * kTileM + row] = acc[i][n];
        }
      }
      auto sum = [&](int i, int j) {
        const float* v = red + (i * BN + j) * kTileM + row;
        float s = v[0];
        for (int r = 1; r < ks; ++r) s += v[(r << own_log) * kTileM];
        return s;
      };
      if (MODE == 1) {
        const bool in = wrow < p.N;
#pragma unroll 2
        for (int j = 0; j < mine; ++j) {
          const float h = in ? silu_f32(sum(0, j)) * sum(1, j) : 0.0f;
          red[j * kTileM + row] = h;  // over this row's first sum, just read
          // positive fp32 numbers order like their bits; a NaN takes no part
          const uint32_t m = __reduce_max_sync(0xffffffffu, h == h ? __float_as_uint(fabsf(h)) : 0u);
          if (lane == 0) s_amax[un & 1][q][j] = __uint_as_float(m);
        }
        named_bar(1, 128);
#pragma unroll 2
        for (int j = 0; j < mine; ++j) {
          const float(*am)[BN] = s_amax[un & 1];
          const QuantScale qs = quant_scale(fmaxf(fmaxf(am[0][j], am[1][j]), fmaxf(am[2][j], am[3][j])));
          const int64_t hr = (int64_t)t.b * p.g.BN + n0 + j;
          if (in) static_cast<uint8_t*>(p.out)[hr * p.out_ld + wrow] = quant1(red[j * kTileM + row], qs);
          if (row == 0) p.hs[hr * nwb + t.m] = qs.s;
        }
      } else {
#pragma unroll 2
        for (int j = 0; j < mine; ++j) {
          const int n = n0 + j;
          const int r = MODE == 2 ? __shfl_sync(0xffffffffu, sid, n & 31) : t.b * BN + n;
          const float v = sum(0, j);
          if (wrow >= p.N) continue;
          const int64_t o = (int64_t)r * p.out_ld + wrow;
          if (MODE == 0 && p.out_f32) static_cast<float*>(p.out)[o] = v;
          else static_cast<uint16_t*>(p.out)[o] = (uint16_t)f32_bf16(v);
        }
      }
      ++un;
    }
  } else if (MODE == 1 && warp >= 8) {
    // -------------------------------------------- token gather (as above)
    const int g = threadIdx.x - 256;
    const int c = g & 7, n = g >> 3;
    int s = 0, ph = 0;  // the next stage; times around the ring
    for (int u = worker, ui = 0; u < total; u += nworkers, ++ui) {
      const Unit t = unit_of<MODE, false>(p, utab, ui, u, nb, BN);
      if (t.skip) continue;
      const int tk = n < t.nvalid ? p.g.sorted_ids[(int64_t)t.b * p.g.BN + n] / p.g.k : 0;
      const uint8_t* src = p.x + (int64_t)tk * p.K + c * 16;
#pragma unroll 1
      for (int kb = k_lo; kb < k_hi; ++kb) {
        wait(&empty[s], ~ph & 1);
        if (__any_sync(0xffffffffu, wait.dead())) break;
        const bool in = kb * kBlkK + c * 16 < p.K;
        cp_async16_or_zero(smem_u32(stages + s * kStage + kA * kTileBytes) + n * kBlkK + ((c ^ (n & 7)) << 4),
                           in ? src + kb * kBlkK : src, in);
        cp_async_mbar_arrive(&full[s]);
        if (++s == p.ns) { s = 0; ++ph; }
      }
    }
    cp_async_wait_all();
    if (lane == 0) s_fills[1 + warp - 8] = ph * p.ns + s;
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    if (wait.dead()) {
      if (lane == 0) drain<MODE>(full, p.ns, s_fills, &s_mma_done, p.g.status);
      __syncwarp();
    }
    tc_fence_after();
    tmem_dealloc(tmem_base, kCols);
  }
  // No CTA leaves while another may still send to it: each has waited for all that
  // is sent to it, unless it gave up.  Then it waits until the others have ended
  // or sent theirs too (they get there: every wait on the way is bounded), and
  // for what they sent.
  if (ks > 1 && wait.dead()) {
    cluster_barrier();
    if (awaited) mbar_wait(&rfull[warp & 3], 0, p.g.status);
  }
}

// ------------------------------------------------------------------ launches
constexpr size_t kSmemBudget = 227 * 1024 - 2560;  // beside the kernels' static shared memory
constexpr int kTmN0 = 256, kTmN2 = 128;  // weight rows a tile: dense, down

template <int MODE, typename OT, int TN>
int launch_tm(const Fp8Maps& maps, Fp8Params p, cudaStream_t stream) {
  p.ks_log = 0;
  const size_t fixed = 1024 + 64 * 8 + 16 + (MODE == 0 ? 0 : kMaxUnitsPerCta * sizeof(UnitRec)) +
                       kTmEpi * 32 * stg_row(MODE) + kScSlots * kTmScFloats * 4;
  p.ns = (int)std::min<size_t>(6, (kSmemBudget - fixed) / tm_stage(TN));
  const size_t smem = fixed + (size_t)p.ns * tm_stage(TN);
  int rc = set_max_dynamic_smem(reinterpret_cast<const void*>(fp8_tm_kernel<MODE, OT, TN>), smem,
                                "fp8_tm_kernel: shared memory limit");
  if (rc) return rc;
  const int64_t units = MODE == 0 ? (int64_t)p.mt * p.nt : INT64_MAX;
  launch_kernel(fp8_tm_kernel<MODE, OT, TN>, (int)std::min<int64_t>(num_sms(), units), tm_threads(MODE), smem, stream, maps, p);
  OES_CHECK_LAUNCH("fp8_tm_kernel");
  return OES_OK;
}

// log2 of the CTAs that share a tile: the largest of 8, 4, 2, 1 with every tile
// resident at once (so a cluster has one tile at most, and its sums' barriers and
// buffers are used once) and two blocks of K for each CTA.  Sharing has a cost (the
// cluster's start, the exchange of sums), so fewer than 8 blocks are not shared
// (8 x 1024 x 1024: 4.4 us shared, 4.9 not; 8 x 2048 x 768: 5.0 and 4.4).
// Clusters of 4 and 8 do not fill the GPU's groups of SMs: 17 clusters of 8 ran
// in two turns, 16 x 2176 x 4096 in 9.2 us, where 17 of 4 took 5.9.  Nor are
// tiles shared that take several turns: 64 tokens x 8 of 64 experts took 83 us
// so, 73 with a tile a CTA.  units: the most units the launch can have, known on
// the host.
int k_shares_log(int64_t units, int nkb) {
  if (nkb < 8) return 0;
  const int64_t sms = num_sms();
  for (int l = 3; l > 0; --l)
    if ((units << l) <= (l == 3 ? sms * 3 / 4 : l == 2 ? sms * 7 / 8 : sms) && nkb >= (2 << l)) return l;
  return 0;
}

template <int MODE, int BN>
int launch_wm(const Fp8Maps& maps, Fp8Params p, int64_t units, cudaStream_t stream) {
  constexpr int stage = wm_stage(MODE, BN);
  p.ks_log = k_shares_log(units, p.nkb);
  const int ks = 1 << p.ks_log;
  const size_t fixed = 1024 + (size_t)(MODE == 1 ? 2 : 1) * BN * kTileM * 4 + 64 * 8 + 16 +
                       kMaxUnitsPerCta * sizeof(UnitRec) + kScSlots * wm_sc_floats(MODE, BN) * 4;
  p.ns = (int)std::min<size_t>(12, (kSmemBudget - fixed) / stage);
  const size_t smem = fixed + (size_t)p.ns * stage;
  auto kernel = fp8_wm_kernel<MODE, BN>;
  int rc = set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), smem, "fp8_wm_kernel: shared memory limit");
  if (rc) return rc;
  const int workers = (int)std::min<int64_t>(num_sms() / ks, std::max<int64_t>(units, 1));
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(workers * ks);
  cfg.blockDim = dim3(wm_threads(MODE));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = t_programmatic_launch ? attr : attr + 1;
  cfg.numAttrs = (t_programmatic_launch ? 1 : 0) + (ks > 1 ? 1 : 0);
  cudaLaunchKernelEx(&cfg, kernel, maps, p);
  OES_CHECK_LAUNCH("fp8_wm_kernel");
  return OES_OK;
}

}  // namespace

Fp8Row fp8_row(int H, int I) {
  const int64_t hb = ceil_div(H, kQuantGroup), ib = ceil_div(I, kQuantGroup);
  auto up = [](int64_t n) { return (n + 15) / 16 * 16; };
  Fp8Row r;
  r.w2 = (int64_t)2 * I * H;
  r.s13 = r.w2 + (int64_t)H * I;
  r.s2 = r.s13 + up(2 * ib * hb * 4);
  r.end = r.s2 + up(hb * ib * 4);
  return r;
}

int fp8_gemm_run(const GemmPlan& g, const GemmParams& p1, const GemmParams& p2, cudaStream_t stream) {
  const int64_t blocks = OES_ALIGN_CAPACITY(p1.R, p1.E, p1.BN) / p1.BN;
  Fp8Maps m{};
  Fp8Params p{};
  p.g = p1;
  m.w = g.m1.a;
  p.x = g.f8.xq;
  p.xs = g.f8.xs;
  p.ws = reinterpret_cast<const float*>(p1.pool + g.f8.s13_off);
  p.N = p1.I;
  p.K = p1.H;
  p.nkb = p1.n_kc;
  p.out = g.f8.hq;
  p.out_ld = p1.I;
  p.hs = g.f8.hs;
  int rc = g.tm ? launch_tm<1, uint16_t, 256>(m, p, stream) : launch_wm<1, 16>(m, p, blocks * p1.n_mtiles, stream);
  if (rc) return rc;
  p.g = p2;
  if (g.tm) p.g.n_mtiles = ceil_div(p1.H, kTmN2);
  m.w = g.m2.a;
  m.x = g.m2.b;
  p.xs = g.f8.hs;
  p.ws = reinterpret_cast<const float*>(p1.pool + g.f8.s2_off);
  p.N = p1.H;
  p.K = p1.I;
  p.nkb = p2.n_kc;
  p.out = p2.y;
  p.out_ld = p1.H;
  return g.tm ? launch_tm<2, uint16_t, kTmN2>(m, p, stream) : launch_wm<2, 16>(m, p, blocks * p2.n_mtiles, stream);
}

}  // namespace oes

using namespace oes;

extern "C" int moe_fp8_gemm(const uint8_t* xq, int64_t xq_ld, const float* xs, int T, int K,
                            const uint8_t* wq, int64_t wq_ld, const float* ws, int N, void* out,
                            int dtype, int64_t out_ld, int32_t* status, oes_stream_t stream) {
  OES_REQUIRE(T >= 0 && K >= 1 && N >= 1 && K <= (1 << 24) && N <= (1 << 24),
              "moe_fp8_gemm: bad T=%d N=%d K=%d", T, N, K);
  OES_REQUIRE(dtype == OES_BF16 || dtype == OES_F32, "moe_fp8_gemm: bad dtype %d", dtype);
  if (T == 0) return OES_OK;
  OES_REQUIRE(xq && xs && wq && ws && out, "moe_fp8_gemm: null pointer");
  OES_REQUIRE(xq_ld >= K && wq_ld >= K && out_ld >= N,
              "moe_fp8_gemm: a row stride is smaller than its row");
  OES_REQUIRE(((uintptr_t)xq & 15) == 0 && ((uintptr_t)wq & 15) == 0 && xq_ld % 16 == 0 && wq_ld % 16 == 0,
              "moe_fp8_gemm: xq and wq must be 16-byte aligned with strides of a multiple of 16");
  OES_REQUIRE(((uintptr_t)xs & 3) == 0 && ((uintptr_t)ws & 3) == 0 &&
                  ((uintptr_t)out & (dtype == OES_BF16 ? 1 : 3)) == 0,
              "moe_fp8_gemm: a pointer is not aligned to its type");
  // Weight-major tiles of 16 or 32 rows while they are one wave of CTAs, else
  // token-major ones: 384 x 1536 x 2048 takes 8.9 us weight-major (144 tiles) and
  // 11.2 token-major, 512 rows 14.5 and 11.2; 160 x 4096 x 4096 22.1 and 18.0.
  const bool tm = T > 16 && (int64_t)ceil_div(T, 32) * ceil_div(N, kTileM) > num_sms();
  const int bn = tm ? kTileM : T <= 16 ? 16 : 32;
  Fp8Params p{};
  p.g.status = status;
  p.xs = xs;
  p.ws = ws;
  p.T = T;
  p.N = N;
  p.K = K;
  p.nkb = ceil_div(K, kQuantGroup);
  p.mt = ceil_div(T, bn);
  p.nt = ceil_div(N, tm ? kTmN0 : kTileM);
  OES_REQUIRE((int64_t)p.mt * p.nt <= 0x7FFFFFFF - 4096, "moe_fp8_gemm: too many tiles (T=%d N=%d)", T, N);
  p.out = out;
  p.out_ld = out_ld;
  p.out_f32 = dtype == OES_F32;
  p.vec = ((uintptr_t)out & 15) == 0 && out_ld % (p.out_f32 ? 4 : 8) == 0 && N % (p.out_f32 ? 4 : 8) == 0;
  Fp8Maps m;
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const uint64_t dw[3] = {(uint64_t)K, (uint64_t)N, 1}, sw[2] = {(uint64_t)wq_ld, (uint64_t)wq_ld * N};
  const uint32_t bw[3] = {kBlkK, kTileM, 1};
  int rc = encode_tiled(&m.w, u8, 3, wq, dw, sw, bw, CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc) return rc;
  const uint64_t dx[2] = {(uint64_t)K, (uint64_t)T}, sx[1] = {(uint64_t)xq_ld};
  const uint32_t bx[2] = {kBlkK, (uint32_t)bn};
  if ((rc = encode_tiled(&m.x, u8, 2, xq, dx, sx, bx, CU_TENSOR_MAP_SWIZZLE_128B))) return rc;
  if (tm) return p.out_f32 ? launch_tm<0, float, kTmN0>(m, p, stream) : launch_tm<0, uint16_t, kTmN0>(m, p, stream);
  const int64_t units = (int64_t)p.mt * p.nt;
  return bn == 16 ? launch_wm<0, 16>(m, p, units, stream) : launch_wm<0, 32>(m, p, units, stream);
}
