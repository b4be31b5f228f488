// Matrix products of e4m3 codes with block scales: moe_fp8_gemm, and the
// grouped SwiGLU expert GEMM of moe_grouped_gemm_slots for the FP8 format.
//
//   out[t, n] = sum_b xs[t, b] ws[n / 128, b] sum_{k in b} x[t, k] w[n, k]
//
// over blocks b of 128 along K: the products of codes of one block are summed
// in fp32, scaled, and added to an fp32 accumulator, block after block.
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "fp8_dev.cuh"
#include "gemm_types.h"
#include "internal.h"

namespace oes {
namespace {

// One launch of the product, dense or grouped.
struct Fp8Args {
  GemmParams g;      // grouped: the routing tables, E, S, H, I, ...
  const uint8_t* x;  // codes of the rows (x, or h)
  int64_t x_ld;
  const float* xs;   // [rows, nkb]
  const uint8_t* w;  // dense: codes [N, K]; grouped: section of the expert row 0
  int64_t w_ld;
  const float* ws;   // dense: [ceil(N/128), nkb]; grouped: section of expert row 0
  int T, N, K, nkb;  // T: dense rows
  void* out;         // MODE 0: [T, N]; MODE 1: codes of h; MODE 2: y
  int64_t out_ld;
  int out_f32;
  float* hs;  // MODE 1: scales of h
};

__device__ __forceinline__ void e4m3x4_f32(uint32_t w, float (&f)[4]) {
  uint32_t lo, hi;
  asm("{ .reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b; }"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
  const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<__half2*>(&hi));
  f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}

// The plain kernel: a CTA computes 16 rows x 128 columns on the FP32 units,
// one 128-block of K at a time through shared memory.
// MODE 0 dense, 1 gate and up with SwiGLU and h's codes, 2 down.
constexpr int kRows = 16;
template <int MODE>
__global__ void __launch_bounds__(256) fp8_simple_kernel(const Fp8Args a) {
  pdl_wait();
  constexpr int kW = MODE == 1 ? 2 : 1;
  __shared__ uint32_t sx[kRows][33];
  __shared__ uint32_t sw[kW][32][129];  // [k / 4][column]
  __shared__ int s_row[kRows];          // row of x, or -1
  __shared__ int s_out[kRows];          // row of the output
  const int ntiles = (a.N + 127) / 128;
  const int tile = blockIdx.x % ntiles, piece = blockIdx.x / ntiles;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint8_t* w = a.w;
  const float* ws = a.ws;
  if (MODE == 0) {
    if (tid < kRows) {
      const int t = piece * kRows + tid;
      s_row[tid] = s_out[tid] = t < a.T ? t : -1;
    }
  } else {
    const GemmParams& g = a.g;
    const int b = piece / (g.BN / kRows), off = piece % (g.BN / kRows) * kRows;
    if (b >= *g.n_post_pad / g.BN) return;
    const int e = g.block_expert[b];
    if (e < 0 || e >= g.E) return;
    if (g.filter && g.flags[e] != g.filter) return;
    const int slot = g.e2s[e];
    const bool bad = slot < 0 || slot >= g.S;
    if (tid < kRows) {
      const int64_t i = (int64_t)b * g.BN + off + tid;
      const int r = g.sorted_ids[i];
      s_row[tid] = r < g.R ? (MODE == 1 ? r / g.k : (int)i) : -1;
      s_out[tid] = r < g.R ? (MODE == 1 ? (int)i : r) : -1;
    }
    if (bad) {
      __syncthreads();
      if (MODE == 2) {
        for (int i = tid; i < kRows * 128; i += 256) {
          const int n = tile * 128 + (i & 127);
          if (s_out[i >> 7] >= 0 && n < a.N)
            static_cast<uint16_t*>(a.out)[(int64_t)s_out[i >> 7] * a.out_ld + n] = 0;
        }
        if (tid == 0 && s_out[0] >= 0) set_status(g.status, OES_DEV_BAD_ID);
      }
      return;
    }
    w += (int64_t)slot * g.row_bytes;
    ws = reinterpret_cast<const float*>(reinterpret_cast<const uint8_t*>(ws) + (int64_t)slot * g.row_bytes);
  }
  __syncthreads();
  float acc[kW][2][4] = {};
  for (int kb = 0; kb < a.nkb; ++kb) {
    // K is read four codes a load where that stays inside a row (strides are
    // multiples of 16), the rest of a block is zero
    auto word = [&](const uint8_t* row, int k) {
      uint32_t v = 0;
      if (k + 4 <= a.K) v = *reinterpret_cast<const uint32_t*>(row + k);
      else
        for (int i = 0; i < 4; ++i)
          if (k + i < a.K) v |= (uint32_t)row[k + i] << (8 * i);
      return v;
    };
    for (int i = tid; i < kRows * 32; i += 256) {
      const int r = s_row[i >> 5];
      sx[i >> 5][i & 31] = r >= 0 ? word(a.x + r * a.x_ld, kb * 128 + (i & 31) * 4) : 0u;
    }
    for (int i = tid; i < kW * 128 * 32; i += 256) {
      const int q = i >> 12, c = (i >> 5) & 127, n = tile * 128 + c;
      sw[q][i & 31][c] = n < a.N ? word(w + ((int64_t)q * a.N + n) * a.w_ld, kb * 128 + (i & 31) * 4) : 0u;
    }
    __syncthreads();
    float part[kW][2][4] = {};
    for (int k4 = 0; k4 < 32; ++k4) {
      float xv[2][4];
      e4m3x4_f32(sx[2 * warp][k4], xv[0]);
      e4m3x4_f32(sx[2 * warp + 1][k4], xv[1]);
#pragma unroll
      for (int q = 0; q < kW; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float wv[4];
          e4m3x4_f32(sw[q][k4][lane + 32 * j], wv);
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) part[q][t][j] = fmaf(xv[t][i], wv[i], part[q][t][j]);
        }
    }
#pragma unroll
    for (int q = 0; q < kW; ++q) {
      const float sb = ws[((int64_t)q * ntiles + tile) * a.nkb + kb];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int r = s_row[2 * warp + t];
        const float sc = r >= 0 ? a.xs[(int64_t)r * a.nkb + kb] * sb : 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[q][t][j] = fmaf(part[q][t][j], sc, acc[q][t][j]);
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int r = s_out[2 * warp + t];
    if (r < 0) continue;  // the whole warp
    float h[4], m = 0.0f;
    if (MODE == 1) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[j] = tile * 128 + lane + 32 * j < a.N ? silu_f32(acc[0][t][j]) * acc[kW - 1][t][j] : 0.0f;
        m = fmaxf(m, fabsf(h[j]));
      }
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    const QuantScale qs = quant_scale(m);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = tile * 128 + lane + 32 * j;
      if (n >= a.N) continue;
      const int64_t o = (int64_t)r * a.out_ld + n;
      if (MODE == 1) static_cast<uint8_t*>(a.out)[o] = quant1(h[j], qs);
      else if (MODE == 0 && a.out_f32) static_cast<float*>(a.out)[o] = acc[0][t][j];
      else static_cast<uint16_t*>(a.out)[o] = (uint16_t)f32_bf16(acc[0][t][j]);
    }
    if (MODE == 1 && lane == 0) a.hs[(int64_t)r * ntiles + tile] = qs.s;
  }
}

template <int MODE>
int launch_simple(const Fp8Args& a, int64_t pieces, cudaStream_t stream) {
  const int64_t grid = pieces * ceil_div(a.N, 128);
  OES_REQUIRE(grid <= 0x7FFFFFFF, "FP8 product: too many tiles");
  launch_kernel(fp8_simple_kernel<MODE>, dim3((unsigned)grid), 256, 0, stream, a);
  OES_CHECK_LAUNCH("fp8_simple_kernel");
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
  const int64_t cap = OES_ALIGN_CAPACITY(p1.R, p1.E, p1.BN);
  Fp8Args a{};
  a.g = p1;
  a.x = g.f8.xq;
  a.x_ld = p1.H;
  a.xs = g.f8.xs;
  a.w = p1.pool;
  a.w_ld = p1.H;
  a.ws = reinterpret_cast<const float*>(p1.pool + g.f8.s13_off);
  a.N = p1.I;
  a.K = p1.H;
  a.nkb = p1.n_kc;
  a.out = g.f8.hq;
  a.out_ld = p1.I;
  a.hs = g.f8.hs;
  int rc = launch_simple<1>(a, cap / kRows, stream);
  if (rc) return rc;
  a.g = p2;
  a.x = g.f8.hq;
  a.x_ld = p1.I;
  a.xs = g.f8.hs;
  a.w = p1.pool + g.f8.w2_off;
  a.w_ld = p1.I;
  a.ws = reinterpret_cast<const float*>(p1.pool + g.f8.s2_off);
  a.N = p1.H;
  a.K = p1.I;
  a.nkb = p2.n_kc;
  a.out = p2.y;
  a.out_ld = p1.H;
  return launch_simple<2>(a, cap / kRows, stream);
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
  Fp8Args a{};
  a.x = xq;
  a.x_ld = xq_ld;
  a.xs = xs;
  a.w = wq;
  a.w_ld = wq_ld;
  a.ws = ws;
  a.T = T;
  a.N = N;
  a.K = K;
  a.nkb = ceil_div(K, kQuantGroup);
  a.out = out;
  a.out_ld = out_ld;
  a.out_f32 = dtype == OES_F32;
  a.g.status = status;
  return launch_simple<0>(a, ceil_div(T, kRows), stream);
}
