// moe_int8_gemm: matrix products of 8-bit integer rows, a scale for each row of
// both sides:
//
//   out[t, n] = xs[t] ws[n] sum_k x[t, k] w[n, k]
//
// GB300's tensor cores have no fast integer products, and need none here: f16
// holds every 8-bit integer exactly, its products are at most 2^14 ((-128)^2) and exact
// in the tensor core, and fp32 sums of up to 1024 of them are at most 2^24, up to which
// fp32 holds every integer.  So the sums of at most 1024 of K (kDrainK, and no more:
// 1024 (-128)^2 is 2^24) come from f16 matrix instructions and are added up as 32-bit
// integers: the sum is the integer, whatever the order, at the f16 rate.
//
//   int8_stream_kernel  few rows: warps stream the weights through queues of their
//                       own (as in few_tokens.cu) into warp-wide instructions, x
//                       stands in shared memory as f16.  One launch, and the weights
//                       are read once as they are.
//   int8_tm_kernel      more rows: 128 rows x 256, 128 or 64 weight rows a tile on
//                       tcgen05, operands by TMA from f16 copies of both that
//                       int8_to_f16_kernel leaves in the workspace (4096 and 8192
//                       rows of 4096: 20 us).
//   int8_pair_kernel    the same for the largest: 256 x 256 a pair of SMs; 4096 x 4096
//                       x 8192 159 us, 1.73 PFLOP/s, 1.52 with the copies.
#include <algorithm>

#include "common.cuh"
#include "fp8_dev.cuh"
#include "tc_dev.cuh"
#include "warp_mma.cuh"

namespace oes {
namespace {

// ================================================================= few rows
// A CTA takes 8 NG tokens and rows_cta rows of w.  Its W warps are W >> wk_log
// groups; a group takes 16 weight rows (one side of the matrix instruction) at a time and
// shares their K range.  Weights go through queues of each lane's own, codes as they are,
// and become f16 on their way to the instruction.  The tokens stand in shared memory as f16, in
// two chunks of K; where K has more, each group has one tile of rows, and chunk after
// chunk is loaded into registers under the products of the chunk two before it.
constexpr int kDrainK = 1024;  // of K in one fp32 sum
static_assert(kDrainK * 128 * 128 <= 1 << 24, "integers that fp32 holds");
constexpr int kStepK = 128;
static_assert(kDrainK % kStepK == 0, "whole steps in a sum");
constexpr int kEntry = 2048;    // 16 rows of a step
constexpr int kTokensMost = 32;  // of a CTA

__host__ __device__ constexpr int chunk_steps(int ng) { return 32 / ng; }  // a chunk is 32 KB of codes

struct StreamArgs {
  const int8_t* x;
  int64_t x_ld;
  const float* xs;
  const int8_t* w;
  int64_t w_ld;
  const float* ws;
  int T, K, N;
  void* out;
  int64_t out_ld;
  int rows_cta, wk_log;  // weight rows a CTA owns; 2^wk_log warps share a tile's K range
  int x_row;             // bytes of a token's row of a chunk in shared memory
};

template <int NG, typename OT, int W, int kQueue>
__global__ void __launch_bounds__(W * 32, 1) int8_stream_kernel(const StreamArgs p) {
  constexpr int kSteps = chunk_steps(NG), kThreads = W * 32;
  constexpr int kHold = 8 * NG * kSteps * kStepK / (16 * kThreads);  // 16 codes each: a thread's share of a chunk
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t queue = smem_u32(smem + warp * (kQueue * kEntry)) + lane * 16;
  uint8_t* xs = smem + W * kQueue * kEntry;             // [2 chunks][8 NG][x_row]
  int32_t* part = reinterpret_cast<int32_t*>(xs);       // afterwards [warp][lane][4 NG]
  const int wk = warp & ((1 << p.wk_log) - 1), wm = warp >> p.wk_log, groups = W >> p.wk_log, share = 1 << p.wk_log;
  const int ns = (p.K + kStepK - 1) / kStepK, chunks = (ns + kSteps - 1) / kSteps;
  const int row_lo = blockIdx.x * p.rows_cta, row_hi = min(p.N, row_lo + p.rows_cta);
  const int tok0 = blockIdx.y * 8 * NG, toks = min(8 * NG, p.T - tok0);
  __shared__ float s_xs[kTokensMost], s_ws[W * 16];  // scales, where warps share tiles
  pdl_begin();

  // The next step to copy: of the tile at row ct, chunk cc, step cs.  A chunk's steps
  // go round the group's warps.
  int ct = row_lo + wm * 16, cc = 0, cs = wk, at = 0;
  const int8_t* r0 = p.w;
  bool ok0 = false, ok1 = false;
  auto steps_of = [&](int c) { return min(kSteps, ns - c * kSteps); };
  auto set_rows = [&]() {
    r0 = p.w + (int64_t)(ct + g) * p.w_ld + 16 * t;
    ok0 = ct + g < row_hi;
    ok1 = ct + g + 8 < row_hi;
  };
  auto skip_empty = [&]() {  // to the warp's next step
    while (ct < row_hi && cs >= steps_of(cc)) {
      cs = wk;
      if (++cc == chunks) {
        cc = 0;
        ct += 16 * groups;
        set_rows();
      }
    }
  };
  set_rows();
  skip_empty();
  auto copy_next = [&]() {
    if (ct < row_hi) {
      const int k = (cc * kSteps + cs) * kStepK;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int o = k + hh * 64, n = max(0, min(16, p.K - o - 16 * t));
        cp_async16_part(queue + at * kEntry + hh * 1024, ok0 && n > 0 ? r0 + o : p.w, ok0 ? n : 0);
        cp_async16_part(queue + at * kEntry + hh * 1024 + 512, ok1 && n > 0 ? r0 + 8 * p.w_ld + o : p.w, ok1 ? n : 0);
      }
      cs += share;
      skip_empty();
    }
    cp_async_commit();
    at = (at + 1) % kQueue;
  };
  for (int i = 0; i < kQueue; ++i) copy_next();

  // Chunk c of the tokens: 16 codes a piece, zeros past K (which silence what a weight's
  // row holds there)
  const int per = min(kSteps, ns) * (kStepK / 16);  // pieces of a token's row
  const int tok_0 = tid / per, pc_0 = tid - tok_0 * per, tok_d = kThreads / per, pc_d = kThreads - tok_d * per;
  uint4 held[kHold];
  auto load_x = [&](int c) {
    int tok = tok_0, pc = pc_0;
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      const int k = c * kSteps * kStepK + pc * 16;
      held[i] = make_uint4(0u, 0u, 0u, 0u);
      if (tok < toks && k < p.K) {
        const int8_t* src = p.x + (int64_t)(tok0 + tok) * p.x_ld + k;
        if (k + 16 <= p.K) {
          held[i] = __ldg(reinterpret_cast<const uint4*>(src));
        } else {
          uint32_t w[4] = {0u, 0u, 0u, 0u};
          for (int j = 0; k + j < p.K; ++j) w[j >> 2] |= (uint32_t)(uint8_t)src[j] << (8 * (j & 3));
          held[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      tok += tok_d;
      pc += pc_d;
      if (pc >= per) {
        pc -= per;
        ++tok;
      }
    }
  };
  auto store_x = [&](int c) {
    uint8_t* to = xs + (c & 1) * (8 * NG * p.x_row);
    int tok = tok_0, pc = pc_0;
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      if (tok < toks) {
        uint32_t o[8];
        s8x4_f16x4(held[i].x, o[0], o[1]);
        s8x4_f16x4(held[i].y, o[2], o[3]);
        s8x4_f16x4(held[i].z, o[4], o[5]);
        s8x4_f16x4(held[i].w, o[6], o[7]);
        uint4* dst = reinterpret_cast<uint4*>(to + tok * p.x_row + pc * 32);
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
      }
      tok += tok_d;
      pc += pc_d;
      if (pc >= per) {
        pc -= per;
        ++tok;
      }
    }
  };
  load_x(0);
  if (share > 1) {
    if (tid < toks) s_xs[tid] = __ldg(p.xs + tok0 + tid);
    if (tid < row_hi - row_lo) s_ws[tid] = __ldg(p.ws + row_lo + tid);
  }
  store_x(0);
  if (chunks > 1) {
    load_x(1);
    store_x(1);
  }
  __syncthreads();

  uint32_t xb[NG];
#pragma unroll
  for (int n = 0; n < NG; ++n) xb[n] = smem_u32(xs + min(8 * n + g, toks - 1) * p.x_row) + 32 * t;
  auto store_out = [&](int n, int tok, int32_t sum, float xscale, float wscale) {
    const float o = (float)sum * xscale * wscale;
    const int64_t at = (int64_t)(tok0 + tok) * p.out_ld + n;
    if constexpr (sizeof(OT) == 2) static_cast<uint16_t*>(p.out)[at] = (uint16_t)f32_bf16(o);
    else static_cast<float*>(p.out)[at] = o;
  };
  int from = 0;
  int32_t acc[NG][4];
  // the sums of the tile at row0; all warps come here together where chunks are reloaded
  auto tile = [&](int row0) {
    float d[NG][4];  // sums of up to 8 steps (kDrainK), integers of at most 2^24
    int steps_in = 0;
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[n][i] = 0;
        d[n][i] = 0.0f;
      }
    auto drain = [&]() {
#pragma unroll
      for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[n][i] += __float2int_rn(d[n][i]);
          d[n][i] = 0.0f;
        }
    };
    for (int c = 0; c < chunks; ++c) {
      if (c + 2 < chunks) load_x(c + 2);
      const uint32_t xo = (c & 1) * (8 * NG * p.x_row);
      const int steps = row0 < row_hi ? steps_of(c) : 0;
      for (int s = wk; s < steps; s += share) {
        cp_async_wait<kQueue - 1>();
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const uint4 a = lds128(queue + from * kEntry + hh * 1024), b = lds128(queue + from * kEntry + hh * 1024 + 512);
          const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
          uint32_t m[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s8x4_f16x4(aw[i], m[i][0], m[i][2]);
            s8x4_f16x4(bw[i], m[i][1], m[i][3]);
          }
#pragma unroll
          for (int n = 0; n < NG; ++n) {
            const uint32_t xa = xb[n] + xo + s * (2 * kStepK) + hh * 128;
            const uint4 u = lds128(xa), v = lds128(xa + 16);
            mma_16816<true>(d[n], m[0][0], m[0][1], m[0][2], m[0][3], u.x, u.y);
            mma_16816<true>(d[n], m[1][0], m[1][1], m[1][2], m[1][3], u.z, u.w);
            mma_16816<true>(d[n], m[2][0], m[2][1], m[2][2], m[2][3], v.x, v.y);
            mma_16816<true>(d[n], m[3][0], m[3][1], m[3][2], m[3][3], v.z, v.w);
          }
        }
        if (++steps_in == kDrainK / kStepK) {
          drain();
          steps_in = 0;
        }
        from = (from + 1) % kQueue;
        copy_next();
      }
      if (c + 2 < chunks) {
        __syncthreads();  // chunk c has been read by all; chunk c + 1, stored before, may be
        store_x(c + 2);
        if (c + 3 == chunks) __syncthreads();  // no other sync before it is read
      }
    }
    drain();
  };
  const int first = row_lo + wm * 16;
  if (share == 1) {
    float xsc[NG][2];
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) xsc[n][j] = __ldg(p.xs + tok0 + min(8 * n + 2 * t + j, toks - 1));
    int row0 = first;
    do {
      const float w0 = __ldg(p.ws + min(row0 + g, p.N - 1)), w1 = __ldg(p.ws + min(row0 + g + 8, p.N - 1));
      if (row0 < row_hi || chunks > 2) tile(row0);
#pragma unroll
      for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = 8 * n + 2 * t + (i & 1), r = row0 + g + 8 * (i >> 1);
          if (tok < toks && r < row_hi) store_out(r, tok, acc[n][i], xsc[n][i & 1], i < 2 ? w0 : w1);
        }
      row0 += 16 * groups;
    } while (row0 < row_hi);  // once, for all warps, where chunks are reloaded
    return;
  }
  // one tile a group at most: its warps' sums go where the tokens were
  tile(first);
  __syncthreads();
  int32_t* mine = part + (warp * 32 + lane) * (4 * NG);
#pragma unroll
  for (int n = 0; n < NG; ++n)
    *reinterpret_cast<int4*>(mine + 4 * n) = make_int4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
  __syncthreads();
  // half a warp a token: 16 rows of a tile
  const int r16 = lane & 15;
  for (int m = 0; row_lo + 16 * m < row_hi; ++m)
    for (int tok = 2 * warp + (lane >> 4); tok < toks; tok += 2 * W) {
      const int32_t* v = part + (m * share * 32 + (r16 & 7) * 4 + (tok & 7) / 2) * (4 * NG) + (tok >> 3) * 4 +
                         (r16 >> 3) * 2 + (tok & 1);
      int32_t sum = 0;
      for (int w = 0; w < share; ++w) sum += v[w * 32 * 4 * NG];
      const int r = 16 * m + r16;
      if (row_lo + r < row_hi) store_out(row_lo + r, tok, sum, s_xs[tok], s_ws[r]);
    }
}

// ================================================================ more rows
struct CvtArgs {
  const int8_t* src[2];  // x, w
  int64_t ld[2];
  uint16_t* dst[2];      // rows of Kp values
  int rows0;             // of x
  int64_t rows;          // of both
  int K, Kp;
  int step_r, step_c;    // the chunks of the whole grid, in rows and chunks
};

// Rows of codes to rows of f16, zeros from K to Kp (a multiple of 64): 8 codes a
// thread, so that a warp's loads and stores are each one piece of memory (with 16, whose
// stores are every other 16 bytes, 4096 and 8192 rows of 4096 took 45 us).  kCvt
// chunks a thread are loaded before the first is stored.
constexpr int kCvt = 4;
__global__ void __launch_bounds__(256) int8_to_f16_kernel(const CvtArgs a) {
  pdl_begin();
  const int nc = a.Kp / 8;
  const int64_t first = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  int64_t r = first / nc;
  int c = (int)(first - r * nc);
  while (r < a.rows) {
    uint2 w[kCvt];
    uint16_t* dst[kCvt];
#pragma unroll
    for (int i = 0; i < kCvt; ++i) {
      w[i] = make_uint2(0u, 0u);
      dst[i] = nullptr;
      if (r < a.rows) {
        const int o = r >= a.rows0;
        const int64_t row = o ? r - a.rows0 : r;
        const int8_t* src = a.src[o] + row * a.ld[o] + c * 8;
        dst[i] = a.dst[o] + row * a.Kp + c * 8;
        if (c * 8 + 8 <= a.K) {
          w[i] = __ldg(reinterpret_cast<const uint2*>(src));
        } else {
          uint32_t v[2] = {0u, 0u};
          for (int j = 0; j < 8 && c * 8 + j < a.K; ++j) v[j >> 2] |= (uint32_t)(uint8_t)src[j] << (8 * (j & 3));
          w[i] = make_uint2(v[0], v[1]);
        }
      }
      r += a.step_r;
      c += a.step_c;
      if (c >= nc) {
        c -= nc;
        ++r;
      }
    }
#pragma unroll
    for (int i = 0; i < kCvt; ++i)
      if (dst[i]) {
        uint32_t v[4];
        s8x4_f16x4(w[i].x, v[0], v[1]);
        s8x4_f16x4(w[i].y, v[2], v[3]);
        *reinterpret_cast<uint4*>(dst[i]) = make_uint4(v[0], v[1], v[2], v[3]);
      }
  }
}

constexpr int kTileM = 128;
constexpr int kBlkBytes = 128;        // 64 f16 of K, a pipeline stage's row
constexpr int kDrain = kDrainK / 64;  // stages a TMEM buffer sums
constexpr int kEpiW0 = 4, kEpi = 8;   // epilogue warps: two a TMEM lane quarter
constexpr int kTmThreads = (kEpiW0 + kEpi) * 32;

struct TmMaps {
  CUtensorMap x, w;  // f16 [T][Kp], [N][Kp]
};
struct TmArgs {
  const float* xs;
  const float* ws;
  int T, N, nkb;  // nkb: stages of K
  int mt, nt;
  void* out;
  int64_t out_ld;
  int vec;  // out's rows and their pieces are multiples of 16 bytes
  int ns;
  int32_t* status;
};

// A warp's part of a tile, 32 rows of kCols sums: scaled, and out.  Results leave in
// pieces of 64 bytes of 32 rows, turned around in shared memory (stg, 2 KB) so that whole
// sectors are stored.
template <typename OT, int kCols>
__device__ __forceinline__ void store_tile(const TmArgs& p, const int32_t (&acc)[kCols], uint8_t* stg, int q, int m0,
                                           int n0, int nvalid) {
  const int lane = threadIdx.x & 31, row = q * 32 + lane;
  constexpr int kPer = 64 / (int)sizeof(OT), kVec = 16 / (int)sizeof(OT);
  const float xscale = row < nvalid ? __ldg(p.xs + m0 + row) : 0.0f;
#pragma unroll
  for (int pc = 0; pc < kCols / kPer; ++pc) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        constexpr int kEach = 4 / (int)sizeof(OT);  // values a word
        float v[kEach];
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          const int j = pc * kPer + c * kVec + i * kEach + e;
          v[e] = (float)acc[j] * xscale * __ldg(p.ws + min(n0 + j, p.N - 1));
        }
        if constexpr (sizeof(OT) == 2) w[i] = f32x2_bf16x2(v[0], v[1]);
        else w[i] = __float_as_uint(v[0]);
      }
      *reinterpret_cast<uint4*>(stg + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncwarp();
    if (p.vec && n0 + (pc + 1) * kPer <= p.N) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int rr = 8 * i + (lane >> 2), c = lane & 3;
        const uint8_t* from = stg + rr * 64 + ((c ^ ((rr >> 1) & 3)) << 4);
        if (q * 32 + rr < nvalid)
          *reinterpret_cast<uint4*>(static_cast<OT*>(p.out) + (int64_t)(m0 + q * 32 + rr) * p.out_ld + n0 + pc * kPer + c * kVec) =
              *reinterpret_cast<const uint4*>(from);
      }
    } else {
      // single values, neighbouring lanes neighbouring columns
      constexpr int kRows = 32 / kPer;  // rows at a time
#pragma unroll 4
      for (int i = 0; i < 32; i += kRows) {
        const int rr = i + lane / kPer, e = lane % kPer, col = n0 + pc * kPer + e;
        const OT v = reinterpret_cast<const OT*>(stg + rr * 64 + ((e / kVec ^ ((rr >> 1) & 3)) << 4))[e % kVec];
        if (q * 32 + rr < nvalid && col < p.N) static_cast<OT*>(p.out)[(int64_t)(m0 + q * 32 + rr) * p.out_ld + col] = v;
      }
    }
    __syncwarp();
  }
}

template <typename OT, int TN>
__global__ void __launch_bounds__(kTmThreads, 1)
    int8_tm_kernel(const __grid_constant__ TmMaps maps, const __grid_constant__ TmArgs p) {
  constexpr int kStage = (kTileM + TN) * kBlkBytes;
  constexpr int kBufs = 512 / TN;
  constexpr int kCols = TN / 2;  // columns of an epilogue warp
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* stg_all = stages + p.ns * kStage;  // 2 KB an epilogue warp
  uint64_t* full = reinterpret_cast<uint64_t*>(stg_all + kEpi * 2048);
  uint64_t* empty = full + p.ns;
  uint64_t* tfull = empty + p.ns;
  uint64_t* tempty = tfull + kBufs;
  __shared__ uint32_t s_tmem;
  __shared__ int s_dead, s_fills;
  __shared__ uint64_t s_mma_done;
  const int warp = warp_index(), lane = threadIdx.x & 31;
  Waits<false> wait{p.status, &s_dead};
  if (threadIdx.x == 0) {
    s_dead = s_fills = 0;
    mbar_init(&s_mma_done, 1);
    for (int s = 0; s < p.ns; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < kBufs; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], kEpi);
    }
    fence_mbar_init();
    tma_prefetch_desc(&maps.x);
    tma_prefetch_desc(&maps.w);
  }
  if (warp == 2) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = s_tmem;
  pdl_wait();  // the f16 copies
  const int total = p.mt * p.nt;

  if (warp < kEpiW0) {
    if (TN == 256) regs_dec<sizeof(OT) == 4 ? 56 : 72>();
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- producer
      int s = 0, ph = 0;
      for (int u = blockIdx.x; u < total; u += gridDim.x) {
        // row tiles fastest: the CTAs of a wave share a few weight tiles
        const int m = u % p.mt, n = u / p.mt;
#pragma unroll 1
        for (int kb = 0; kb < p.nkb; ++kb) {
          wait(&empty[s], ~ph & 1);
          if (wait.dead()) break;
          uint8_t* X = stages + s * kStage;
          mbar_arrive_expect_tx(&full[s], kStage);
          tma_load_2d(X, &maps.x, &full[s], kb * 64, m * kTileM);
#pragma unroll
          for (int j = 0; j < TN; j += 64)
            tma_load_2d(X + (kTileM + j) * kBlkBytes, &maps.w, &full[s], kb * 64, n * TN + j);
          if (++s == p.ns) { s = 0; ++ph; }
        }
      }
      s_fills = ph * p.ns + s;
    } else if (warp == 1) {
      // -------------------------------------------------------- MMA issuer
      int s = 0, ph = 0;
      uint32_t it = 0;
      const uint32_t idesc = idesc_f16(0, kTileM, TN);
      const uint64_t desc0 = smem_desc_sw128(smem_u32(stages));
      const bool leader = elect_one();
      for (int u = blockIdx.x; u < total; u += gridDim.x) {
#pragma unroll 1
        for (int kb = 0; kb < p.nkb; ++kb) {
          const uint32_t a = it % kBufs;
          const bool opens = kb % kDrain == 0, closes = (kb + 1) % kDrain == 0 || kb + 1 == p.nkb;
          if (opens) wait(&tempty[a], ((it / kBufs) & 1) ^ 1);
          wait(&full[s], ph);
          tc_fence_after();
          if (leader) {
            const uint64_t xd = desc0 + (uint32_t)(s * (kStage >> 4)), wd = xd + (kTileM * kBlkBytes >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_f16(tmem_base + a * TN, xd + 2 * kk, wd + 2 * kk, idesc, opens && kk == 0 ? 0u : 1u);
            tc_commit(&empty[s]);
            if (closes) tc_commit(&tfull[a]);
          }
          __syncwarp();
          if (closes) ++it;
          if (++s == p.ns) { s = 0; ph ^= 1; }
        }
      }
      if (leader) tc_commit(&s_mma_done);
    }
  } else {
    if (TN == 256) regs_inc<sizeof(OT) == 4 ? 224 : 216>();
    // ---------------------------------------------------------- epilogue
    const int q = warp & 3, half = (warp - kEpiW0) >> 2;  // 32 q + lane: TMEM lane and row of the tile
    uint8_t* const stg = stg_all + (warp - kEpiW0) * 2048;
    const int nd = (p.nkb + kDrain - 1) / kDrain;
    uint32_t it = 0;
    for (int u = blockIdx.x; u < total; u += gridDim.x) {
      const int m0 = u % p.mt * kTileM, n0 = u / p.mt * TN + half * kCols;
      const int nvalid = min(kTileM, p.T - m0);
      const bool on = q * 32 < nvalid && n0 < p.N;
      int32_t acc[kCols];
#pragma unroll
      for (int j = 0; j < kCols; ++j) acc[j] = 0;
#pragma unroll 1
      for (int d = 0; d < nd; ++d, ++it) {
        const uint32_t a = it % kBufs;
        wait(&tfull[a], (it / kBufs) & 1);
        tc_fence_after();
        if (on) {
          const uint32_t tl = tmem_base + ((uint32_t)(q * 32) << 16) + a * TN + half * kCols;
#pragma unroll
          for (int c = 0; c < kCols / 32; ++c) {
            uint32_t r[32];
            tmem_ld_32(tl + c * 32, r);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[c * 32 + j] += __float2int_rn(__uint_as_float(r[j]));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[a]);
      }
      if (!on) continue;
      store_tile<OT, kCols>(p, acc, stg, q, m0, n0, nvalid);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    if (wait.dead()) {
      // a wait gave up: no copy and no MMA of the CTA outlives its shared memory and TMEM
      if (lane == 0) {
        const int fills = *(volatile int*)&s_fills;
        for (int i = max(0, fills - p.ns); i < fills; ++i) mbar_wait(&full[i % p.ns], (i / p.ns) & 1, p.status);
        mbar_wait(&s_mma_done, 0, p.status);
      }
      __syncwarp();
    }
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// ----- two SMs on one tile
// 256 rows x 256 weight rows a pair of CTAs.  A matrix instruction of the pair
// (cta_group::2, issued by the CTA of rank 0) takes 128 rows of x and 128 weight rows from each
// one's shared memory and leaves 128 x 256 sums in each one's tensor memory, so that a
// stage is 32 KB a CTA where a tile of its own takes 48: one SM's tile moved 96 bytes a
// clock into its shared memory and as many out of it, and the tensor pipe was active for 72 %.
//
// Both CTAs' loads are counted by the barriers of rank 0, which issues; the instructions'
// completion is told to both.  (With the loads counted by barriers of each CTA's own and
// passed on by a thread of rank 1, whose releasing arrivals took 0.8 us each, 4096 x 8192 x
// 4096 took 442 us.)
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void pair_mma_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// a box into this CTA's shared memory, its bytes counted by a barrier of either CTA
__device__ __forceinline__ void pair_load_2d(void* dst, const CUtensorMap* m, uint32_t cluster_bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, "
      "%4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(cluster_bar), "r"(x), "r"(y)
      : "memory");
}
// one arrival at this barrier in both CTAs once all earlier instructions are done
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

template <typename OT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kTmThreads, 1)
    int8_pair_kernel(const __grid_constant__ TmMaps maps, const __grid_constant__ TmArgs p) {
  constexpr int kTile = 256, kStage = 2 * kTileM * kBlkBytes, kBufs = 2, kCols = 128;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* stg_all = stages + p.ns * kStage;  // 2 KB an epilogue warp
  uint64_t* full = reinterpret_cast<uint64_t*>(stg_all + kEpi * 2048);
  uint64_t* empty = full + p.ns;
  uint64_t* tfull = empty + p.ns;
  uint64_t* tempty = tfull + kBufs;  // rank 0: both CTAs' warps have read
  __shared__ uint32_t s_tmem;
  __shared__ int s_dead, s_fills;
  __shared__ uint64_t s_mma_done;
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  Waits<false> wait{p.status, &s_dead};
  if (threadIdx.x == 0) {
    s_dead = s_fills = 0;
    mbar_init(&s_mma_done, 1);
    for (int s = 0; s < p.ns; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < kBufs; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * kEpi);
    }
    fence_mbar_init();
    tma_prefetch_desc(&maps.x);
    tma_prefetch_desc(&maps.w);
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  __syncthreads();
  cluster_barrier();  // the other CTA's barriers and tensor memory are there
  tc_fence_after();
  const uint32_t tmem_base = s_tmem;
  pdl_wait();  // the f16 copies
  const int total = p.mt * p.nt, first = blockIdx.x >> 1, step = gridDim.x >> 1;

  if (warp < kEpiW0) {
    regs_dec<sizeof(OT) == 4 ? 56 : 72>();
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- producer
      int s = 0, ph = 0;
      for (int u = first; u < total; u += step) {
        const int m = (u % p.mt) * kTile + rank * kTileM, n = (u / p.mt) * kTile + rank * 128;
#pragma unroll 1
        for (int kb = 0; kb < p.nkb; ++kb) {
          wait(&empty[s], ~ph & 1);
          if (wait.dead()) break;
          // Rank 0 expects both CTAs' bytes.  Rank 1's may come first: its stage was released
          // with rank 0's, and the phase does not end before rank 0's arrival.
          uint8_t* X = stages + s * kStage;
          const uint32_t bar = map_rank(smem_u32(&full[s]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kStage);
          pair_load_2d(X, &maps.x, bar, kb * 64, m);
          pair_load_2d(X + kTileM * kBlkBytes, &maps.w, bar, kb * 64, n);
          pair_load_2d(X + (kTileM + 64) * kBlkBytes, &maps.w, bar, kb * 64, n + 64);
          if (++s == p.ns) { s = 0; ++ph; }
        }
      }
      s_fills = ph * p.ns + s;
    } else if (warp == 1 && rank == 0) {
      // -------------------------------------------------------- MMA issuer
      int s = 0, ph = 0;
      uint32_t it = 0;
      const uint32_t idesc = idesc_f16(0, kTile, kTile);
      const uint64_t desc0 = smem_desc_sw128(smem_u32(stages));
      const bool leader = elect_one();
      for (int u = first; u < total; u += step) {
#pragma unroll 1
        for (int kb = 0; kb < p.nkb; ++kb) {
          const uint32_t a = it % kBufs;
          const bool opens = kb % kDrain == 0, closes = (kb + 1) % kDrain == 0 || kb + 1 == p.nkb;
          if (opens) wait(&tempty[a], ((it / kBufs) & 1) ^ 1);
          wait(&full[s], ph);
          tc_fence_after();
          // Once a wait has given up nothing is released, so that rank 1's loads stop too.
          if (leader && !wait.dead()) {
            const uint64_t xd = desc0 + (uint32_t)(s * (kStage >> 4)), wd = xd + (kTileM * kBlkBytes >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              pair_mma_f16(tmem_base + a * kTile, xd + 2 * kk, wd + 2 * kk, idesc, opens && kk == 0 ? 0u : 1u);
            pair_commit(&empty[s]);
            if (closes) pair_commit(&tfull[a]);
          }
          __syncwarp();
          if (closes) ++it;
          if (++s == p.ns) { s = 0; ph ^= 1; }
        }
      }
      if (leader) pair_commit(&s_mma_done);
    }
  } else {
    regs_inc<sizeof(OT) == 4 ? 224 : 216>();
    // ---------------------------------------------------------- epilogue
    const int q = warp & 3, half = (warp - kEpiW0) >> 2;
    uint8_t* const stg = stg_all + (warp - kEpiW0) * 2048;
    const int nd = (p.nkb + kDrain - 1) / kDrain;
    uint32_t it = 0;
    for (int u = first; u < total; u += step) {
      const int m0 = (u % p.mt) * kTile + rank * kTileM, n0 = (u / p.mt) * kTile + half * kCols;
      const int nvalid = min(kTileM, p.T - m0);
      const bool on = q * 32 < nvalid && n0 < p.N;
      int32_t acc[kCols];
#pragma unroll
      for (int j = 0; j < kCols; ++j) acc[j] = 0;
#pragma unroll 1
      for (int d = 0; d < nd; ++d, ++it) {
        const uint32_t a = it % kBufs;
        wait(&tfull[a], (it / kBufs) & 1);
        tc_fence_after();
        if (on) {
          const uint32_t tl = tmem_base + ((uint32_t)(q * 32) << 16) + a * kTile + half * kCols;
#pragma unroll
          for (int c = 0; c < kCols / 32; ++c) {
            uint32_t r[32];
            tmem_ld_32(tl + c * 32, r);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[c * 32 + j] += __float2int_rn(__uint_as_float(r[j]));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (rank == 0) mbar_arrive(&tempty[a]);
          else arrive_remote(map_rank(smem_u32(&tempty[a]), 0));
        }
      }
      if (on) store_tile<OT, kCols>(p, acc, stg, q, m0, n0, nvalid);
    }
  }

  tc_fence_before();
  __syncthreads();
  // No copy outlives the shared memory it goes to, no instruction the tensor memory or what
  // it reads, no arrival the CTA it goes to.
  if (warp == 2 && lane == 0) mbar_wait(&s_mma_done, 0, p.status);
  __syncwarp();
  cluster_barrier();
  if (rank == 0 && threadIdx.x == 0) {
    int theirs, their_dead;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(theirs) : "r"(map_rank(smem_u32(&s_fills), 1)));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(their_dead) : "r"(map_rank(smem_u32(&s_dead), 1)));
    if (s_dead || their_dead) {
      // A wait gave up, and one producer may have stopped before the other: what a phase
      // of the last ns is short of is made up, then its bytes are waited for.
      const int mine = s_fills, most = max(mine, theirs);
      for (int i = max(0, most - p.ns); i < most; ++i) {
        uint64_t* bar = &full[i % p.ns];
        if (i >= mine) mbar_arrive_expect_tx(bar, kStage);
        if (i >= theirs)
          asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(kStage)
                       : "memory");
        mbar_wait(bar, (i / p.ns) & 1, p.status);
      }
    }
  }
  __syncthreads();
  cluster_barrier();
  if (warp == 2) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem_base) : "memory");
  }
}

// ------------------------------------------------------------------ launches
constexpr size_t kSmemMost = 227 * 1024 - 2048;  // beside the kernels' static shared memory

// How few rows are cut up: NG groups of 8 tokens a CTA, weight rows a CTA, warps that
// share a tile.  false: the tensor-memory kernel's.  A function of the sizes alone (the
// workspace's size follows it, also where there is no GPU).
constexpr int kSms = 152;
struct Cut {
  int ng, tiles, rows, warps, wk_log;
};
bool stream_cut(int T, int K, int N, Cut* c) {
  c->ng = T <= 8 ? 1 : T <= 16 ? 2 : 4;
  c->tiles = ceil_div(T, 8 * c->ng);
  if (c->tiles > kSms) return false;
  c->rows = ceil_div(N, kSms / c->tiles);
  if (c->tiles > 1) c->rows = ceil_div(c->rows, 16) * 16;
  // Short rows are done before 16 warps have set themselves up: 200 x 768 x 2048 takes 6.2
  // us with 8 and 8.1 with 16, 1024 x 512 x 512 5.6 and 7.5, 1 x 2048 x 1536 3.5 and 3.2,
  // 128 x 2048 x 2048 10.9 and 9.8.
  c->warps = K <= 1024 ? 8 : 16;
  int groups = 1;  // of warps, one for each tile of 16 rows, at most all
  while (groups < c->warps && groups * 16 < c->rows) groups *= 2;
  c->wk_log = 0;
  for (int g = groups; g < c->warps; g *= 2) ++c->wk_log;
  const int64_t chunks = ceil_div(ceil_div(K, kStepK), chunk_steps(c->ng));
  if (chunks > 2 && groups * 16 < c->rows) return false;  // chunks are loaded again for one tile only
  // Both ways' times, in us, as they were measured over 30 sizes.  The stream: 3.9 and
  // 0.09 for each step (16 weight rows x 128 of K) of a CTA.  The tensor-memory kernel:
  // its two launches, the f16 copies' 3 bytes a code, 0.13 for each 64 of K.
  //   rows x K x N         stream  tensor       rows x K x N       stream  tensor
  //   32 x 4096 x 8192      17.5    37.7        200 x 768 x 2048     6.2     8.9
  //   64 x 512 x 512         4.0     6.1        256 x 4096 x 4096   36.5    29.3
  //   128 x 4096 x 4096     23.4    29.0        1024 x 512 x 512     5.6     7.2
  //   128 x 2048 x 2048      9.7    14.8        512 x 1024 x 1024    9.8     9.6
  const double stream = 3.9 + 0.09 * ceil_div(c->rows, 16) * ceil_div(K, kStepK);
  const double tensor = 5.8 + 1.2 * (0.13 * ceil_div(K, 64) + 3.0 * ((double)T + N) * K / 4.5e6);
  return stream <= tensor;
}
int stream_x_row(int K, int ng) { return std::min(ceil_div(K, kStepK), chunk_steps(ng)) * kStepK * 2 + 16; }
bool few_rows(int T, int K, int N) {
  Cut c;
  return T > 0 && stream_cut(T, K, N, &c);
}
int64_t padded_k(int K) { return ceil_div64(K, 64) * 64; }
size_t align256(size_t n) { return (n + 255) / 256 * 256; }

template <int NG, typename OT, int W, int kQueue>
int launch_stream_of(const StreamArgs& a, const Cut& c, size_t fixed, cudaStream_t stream) {
  const size_t smem = fixed + W * kQueue * kEntry;
  int rc = set_max_dynamic_smem(reinterpret_cast<const void*>(int8_stream_kernel<NG, OT, W, kQueue>), smem,
                                "int8_stream_kernel: shared memory limit");
  if (rc) return rc;
  launch_kernel(int8_stream_kernel<NG, OT, W, kQueue>, dim3(ceil_div(a.N, c.rows), c.tiles), W * 32, smem, stream, a);
  OES_CHECK_LAUNCH("int8_stream_kernel");
  return OES_OK;
}
template <int NG, typename OT>
int launch_stream(StreamArgs a, const Cut& c, cudaStream_t stream) {
  a.x_row = stream_x_row(a.K, NG);
  a.rows_cta = c.rows;
  a.wk_log = c.wk_log;
  const size_t sums = c.wk_log ? (size_t)c.warps * 32 * 16 * NG : 0;
  const int chunks = ceil_div(ceil_div(a.K, kStepK), chunk_steps(NG));
  const size_t fixed = std::max(sums, (size_t)std::min(chunks, 2) * 8 * NG * a.x_row);
  if (c.warps == 8) return launch_stream_of<NG, OT, 8, 4>(a, c, fixed, stream);
  // as deep a queue as fits
  if (fixed + 16 * 4 * kEntry <= kSmemMost) return launch_stream_of<NG, OT, 16, 4>(a, c, fixed, stream);
  return launch_stream_of<NG, OT, 16, 2>(a, c, fixed, stream);
}

template <typename OT, int TN>
int launch_tm(const TmMaps& maps, TmArgs a, cudaStream_t stream) {
  constexpr int stage = (kTileM + TN) * kBlkBytes;
  const size_t fixed = 1024 + kEpi * 2048 + 64 * 8;
  a.ns = (int)std::min<size_t>(8, (kSmemMost - fixed) / stage);
  const size_t smem = fixed + (size_t)a.ns * stage;
  int rc = set_max_dynamic_smem(reinterpret_cast<const void*>(int8_tm_kernel<OT, TN>), smem,
                                "int8_tm_kernel: shared memory limit");
  if (rc) return rc;
  launch_kernel(int8_tm_kernel<OT, TN>, std::min(num_sms(), a.mt * a.nt), kTmThreads, smem, stream, maps, a);
  OES_CHECK_LAUNCH("int8_tm_kernel");
  return OES_OK;
}

template <typename OT>
int launch_pair(const TmMaps& maps, TmArgs a, cudaStream_t stream) {
  constexpr int stage = 2 * kTileM * kBlkBytes;
  const size_t fixed = 1024 + kEpi * 2048 + 64 * 8;
  a.ns = (int)std::min<size_t>(8, (kSmemMost - fixed) / stage);
  const size_t smem = fixed + (size_t)a.ns * stage;
  int rc = set_max_dynamic_smem(reinterpret_cast<const void*>(int8_pair_kernel<OT>), smem,
                                "int8_pair_kernel: shared memory limit");
  if (rc) return rc;
  launch_kernel(int8_pair_kernel<OT>, 2 * std::min(num_sms() / 2, a.mt * a.nt), kTmThreads, smem, stream, maps, a);
  OES_CHECK_LAUNCH("int8_pair_kernel");
  return OES_OK;
}

template <typename OT>
int run_stream(const StreamArgs& a, const Cut& c, cudaStream_t stream) {
  return c.ng == 1 ? launch_stream<1, OT>(a, c, stream) : c.ng == 2 ? launch_stream<2, OT>(a, c, stream)
                                                                    : launch_stream<4, OT>(a, c, stream);
}

bool sizes_ok(int T, int K, int N) {
  return T >= 0 && T <= (1 << 28) && K >= 1 && K <= 65536 && N >= 1 && N <= (1 << 24);
}

}  // namespace
}  // namespace oes

using namespace oes;

extern "C" size_t moe_int8_gemm_workspace_size(int T, int K, int N) {
  if (!sizes_ok(T, K, N) || T == 0 || few_rows(T, K, N)) return 0;
  return align256((size_t)T * padded_k(K) * 2) + align256((size_t)N * padded_k(K) * 2);
}

extern "C" int moe_int8_gemm(const int8_t* xq, int64_t xq_ld, const float* xs, int T, int K, const int8_t* wq,
                             int64_t wq_ld, const float* ws, int N, void* out, int dtype, int64_t out_ld,
                             void* workspace, size_t workspace_bytes, int32_t* status, oes_stream_t stream) {
  OES_REQUIRE(sizes_ok(T, K, N), "moe_int8_gemm: bad T=%d N=%d K=%d", T, N, K);
  OES_REQUIRE(dtype == OES_BF16 || dtype == OES_F32, "moe_int8_gemm: bad dtype %d", dtype);
  if (T == 0) return OES_OK;
  OES_REQUIRE(xq && xs && wq && ws && out, "moe_int8_gemm: null pointer");
  OES_REQUIRE(xq_ld >= K && wq_ld >= K && out_ld >= N, "moe_int8_gemm: a row stride is smaller than its row");
  OES_REQUIRE(((uintptr_t)xq & 15) == 0 && ((uintptr_t)wq & 15) == 0 && xq_ld % 16 == 0 && wq_ld % 16 == 0,
              "moe_int8_gemm: xq and wq must be 16-byte aligned with strides of a multiple of 16");
  OES_REQUIRE((((uintptr_t)xs | (uintptr_t)ws | (uintptr_t)status) & 3) == 0 &&
                  ((uintptr_t)out & (dtype == OES_BF16 ? 1 : 3)) == 0,
              "moe_int8_gemm: a pointer is not aligned to its type");
  const size_t need = moe_int8_gemm_workspace_size(T, K, N);
  OES_REQUIRE(need == 0 || (workspace && ((uintptr_t)workspace & 255) == 0 && workspace_bytes >= need),
              "moe_int8_gemm: a 256-byte aligned workspace of %zu bytes is required", need);
  Cut cut;
  if (stream_cut(T, K, N, &cut)) {
    StreamArgs a{xq, xq_ld, xs, wq, wq_ld, ws, T, K, N, out, out_ld, 0, 0, 0};
    return dtype == OES_BF16 ? run_stream<uint16_t>(a, cut, stream) : run_stream<float>(a, cut, stream);
  }
  const int64_t Kp = padded_k(K);
  uint16_t* xf = static_cast<uint16_t*>(workspace);
  uint16_t* wf = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(workspace) + align256((size_t)T * Kp * 2));
  TmArgs a{};
  a.xs = xs;
  a.ws = ws;
  a.T = T;
  a.N = N;
  a.nkb = (int)(Kp / 64);
  a.mt = ceil_div(T, kTileM);
  // Weight rows a tile: the widest whose tiles leave at most a third of the SMs idle.
  // 1024 x 4096 x 4096 takes 42.7 us with 256 (128 tiles), 52 with 128 and 77 with 64; 512
  // x 2048 x 4096 25.8, 20.4 and 25.7; 256 x 4096 x 4096 39.7, 32.2 and 29.3.
  const int enough = num_sms() * 2 / 3;
  const int tn = (int64_t)a.mt * ceil_div(N, 256) >= enough ? 256 : (int64_t)a.mt * ceil_div(N, 128) >= enough ? 128 : 64;
  a.nt = ceil_div(N, tn);
  OES_REQUIRE((int64_t)a.mt * a.nt <= 0x7FFFFFFF - 4096, "moe_int8_gemm: too many tiles (T=%d N=%d)", T, N);
  a.out = out;
  a.out_ld = out_ld;
  const int vec = dtype == OES_F32 ? 4 : 8;
  a.vec = ((uintptr_t)out & 15) == 0 && out_ld % vec == 0;
  a.status = status;
  TmMaps m;
  const uint64_t dx[2] = {(uint64_t)Kp, (uint64_t)T}, dw[2] = {(uint64_t)Kp, (uint64_t)N}, st[1] = {(uint64_t)Kp * 2};
  const uint32_t bx[2] = {64, kTileM}, bw[2] = {64, 64};
  int rc = encode_tiled(&m.x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, xf, dx, st, bx, CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc) return rc;
  if ((rc = encode_tiled(&m.w, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, wf, dw, st, bw, CU_TENSOR_MAP_SWIZZLE_128B))) return rc;
  CvtArgs c{};
  c.src[0] = xq;
  c.src[1] = wq;
  c.ld[0] = xq_ld;
  c.ld[1] = wq_ld;
  c.dst[0] = xf;
  c.dst[1] = wf;
  c.rows0 = T;
  c.rows = (int64_t)T + N;
  c.K = K;
  c.Kp = (int)Kp;
  const int grid = (int)std::min<int64_t>(ceil_div64(c.rows * (Kp / 8), 256), (int64_t)num_sms() * 8);
  c.step_r = (int)((int64_t)grid * 256 / (Kp / 8));
  c.step_c = (int)((int64_t)grid * 256 % (Kp / 8));
  launch_kernel(int8_to_f16_kernel, grid, 256, 0, stream, c);
  OES_CHECK_LAUNCH("int8_to_f16_kernel");
  // Pairs of SMs where every pair has a tile and K is long: 4096 x 4096 x 8192 takes 181 us,
  // 192 with tiles of one SM, 2048 x 4096 x 4096 66 and 68; 4096 x 768 x 2048 28 and 26.
  if (tn == 256 && K >= 2048 && (int64_t)ceil_div(T, 256) * a.nt >= num_sms() / 2) {
    a.mt = ceil_div(T, 256);
    return dtype == OES_BF16 ? launch_pair<uint16_t>(m, a, stream) : launch_pair<float>(m, a, stream);
  }
  if (tn == 256) return dtype == OES_BF16 ? launch_tm<uint16_t, 256>(m, a, stream) : launch_tm<float, 256>(m, a, stream);
  if (tn == 128) return dtype == OES_BF16 ? launch_tm<uint16_t, 128>(m, a, stream) : launch_tm<float, 128>(m, a, stream);
  return dtype == OES_BF16 ? launch_tm<uint16_t, 64>(m, a, stream) : launch_tm<float, 64>(m, a, stream);
}
