// moe_fp8_quantize: rows of bf16 or fp32, or SwiGLU of such rows, to e4m3
// codes with one fp32 scale for each 128 values (the formulas are in
// fp8_dev.cuh).  Bound by memory traffic: 3 bytes a value from bf16.
#include <algorithm>

#include "common.cuh"
#include "fp8_dev.cuh"
#include "internal.h"

namespace oes {
namespace {

struct QuantArgs {
  const void* x;
  int64_t ld;      // of x, in values
  int64_t up;      // SwiGLU: offset of the up half of a row
  int64_t groups;  // T * nb
  int K, nb;
  int step_t, step_b;  // the groups of the whole grid, in rows and blocks
  uint8_t* q;
  int64_t q_ld;
  float* s;
};

// VEC 8: 16 lanes hold a group, 8 values each.  VEC 1: a warp holds a group,
// value lane + 32 i.  Plain rows of 8 take two groups a turn, both loaded before
// the first is reduced (16384 x 4096 bf16: 44 us, 4.6 TB/s; one at a time 51
// us).  The others do better with one and more threads (4096 x 2047: 9.2 us, two at a
// time 10.4).
template <int VEC, bool SWIGLU, typename XT>
__global__ void __launch_bounds__(256) fp8_quantize_kernel(const QuantArgs a) {
  pdl_begin();
  constexpr int kLanes = VEC == 8 ? 16 : 32;
  constexpr int kPer = kQuantGroup / kLanes;
  constexpr int kTurn = VEC == 8 && !SWIGLU ? 2 : 1;
  const int gl = threadIdx.x & (kLanes - 1);
  const int64_t per_grid = (int64_t)gridDim.x * (blockDim.x / kLanes);
  // every lane of a warp makes the same number of turns (the shuffles below)
  const int64_t first = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / kLanes;
  const int odd = VEC == 8 ? (int)(first & 1) : 0;
  int64_t t = first / a.nb;
  int b = (int)(first - t * a.nb);
  for (int64_t g0 = first - odd; g0 < a.groups; g0 += kTurn * per_grid) {
    float v[kTurn][kPer];
    int64_t row[kTurn];
    int k0[kTurn];
#pragma unroll
    for (int n = 0; n < kTurn; ++n) {
      if (b >= a.nb) {
        b -= a.nb;
        ++t;
      }
      row[n] = t;
      k0[n] = b * kQuantGroup;
      const bool live = g0 + odd + n * per_grid < a.groups;
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[n][i] = 0.0f;
      const XT* xp = static_cast<const XT*>(a.x) + t * a.ld;
      if constexpr (VEC == 8) {
        const int k = k0[n] + gl * 8;
        if (live && k < a.K) {
          load_vals<8>(xp + k, v[n]);
          if (SWIGLU) {
            float u[8];
            load_vals<8>(xp + a.up + k, u);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[n][i] = silu_f32(v[n][i]) * u[i];
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int k = k0[n] + gl + 32 * i;
          if (live && k < a.K) {
            float w[1], u[1];
            load_vals<1>(xp + k, w);
            v[n][i] = w[0];
            if (SWIGLU) {
              load_vals<1>(xp + a.up + k, u);
              v[n][i] = silu_f32(w[0]) * u[0];
            }
          }
        }
      }
      t += a.step_t;
      b += a.step_b;
    }
#pragma unroll
    for (int n = 0; n < kTurn; ++n) {
      const int64_t g = g0 + odd + n * per_grid;
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) m = fmaxf(m, fabsf(v[n][i]));
#pragma unroll
      for (int o = kLanes / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (g >= a.groups) continue;
      const QuantScale qs = quant_scale(m);
      uint8_t* qp = a.q + row[n] * a.q_ld;
      if constexpr (VEC == 8) {
        const int k = k0[n] + gl * 8;
        if (k < a.K)
          *reinterpret_cast<uint2*>(qp + k) = make_uint2(quant4(v[n][0], v[n][1], v[n][2], v[n][3], qs),
                                                         quant4(v[n][4], v[n][5], v[n][6], v[n][7], qs));
      } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int k = k0[n] + gl + 32 * i;
          if (k < a.K) qp[k] = quant1(v[n][i], qs);
        }
      }
      if (gl == 0) a.s[g] = qs.s;
    }
  }
}

template <int VEC, bool SWIGLU, typename XT>
int launch_quant(const QuantArgs& a, cudaStream_t stream) {
  const int per_cta = 256 / (VEC == 8 ? 16 : 32);
  // SwiGLU of rows of 8 has registers for six CTAs an SM: at eight 4096 x 2048 took
  // 12.7 us, at six 11.5 (4096 x 768 4.5 and 4.4)
  const int per_sm = VEC == 8 && SWIGLU ? 6 : 8;
  const int grid = (int)std::min<int64_t>(ceil_div64(a.groups, per_cta), (int64_t)num_sms() * per_sm);
  QuantArgs args = a;
  args.step_t = grid * per_cta / a.nb;
  args.step_b = grid * per_cta % a.nb;
  launch_kernel(fp8_quantize_kernel<VEC, SWIGLU, XT>, grid, 256, 0, stream, args);
  OES_CHECK_LAUNCH("fp8_quantize_kernel");
  return OES_OK;
}

template <int VEC>
int launch_quant_of(const QuantArgs& a, int dtype, int act, cudaStream_t stream) {
  if (act == OES_ACT_SWIGLU)
    return dtype == OES_BF16 ? launch_quant<VEC, true, uint16_t>(a, stream)
                             : launch_quant<VEC, true, float>(a, stream);
  return dtype == OES_BF16 ? launch_quant<VEC, false, uint16_t>(a, stream)
                           : launch_quant<VEC, false, float>(a, stream);
}

}  // namespace

int fp8_quantize(const void* x, int dtype, int64_t x_ld, int T, int K, int act, uint8_t* q,
                 int64_t q_ld, float* scale, cudaStream_t stream) {
  QuantArgs a{};
  a.x = x;
  a.ld = x_ld;
  a.up = K;
  a.K = K;
  a.nb = ceil_div(K, kQuantGroup);
  a.groups = (int64_t)T * a.nb;
  a.q = q;
  a.q_ld = q_ld;
  a.s = scale;
  // eight values a load where rows, both halves and codes are aligned for it
  const int64_t m = dtype == OES_BF16 ? 8 : 4;
  const bool vec = K % 8 == 0 && ((uintptr_t)x & 15) == 0 && x_ld % m == 0 &&
                   ((uintptr_t)q & 7) == 0 && q_ld % 8 == 0;
  return vec ? launch_quant_of<8>(a, dtype, act, stream) : launch_quant_of<1>(a, dtype, act, stream);
}

}  // namespace oes

using namespace oes;

extern "C" int moe_fp8_quantize(const void* x, int dtype, int64_t x_ld, int T, int K, int act,
                                uint8_t* q, int64_t q_ld, float* scale, oes_stream_t stream) {
  OES_REQUIRE(T >= 0 && K >= 1 && K <= (1 << 28), "moe_fp8_quantize: bad T=%d K=%d", T, K);
  OES_REQUIRE(dtype == OES_BF16 || dtype == OES_F32, "moe_fp8_quantize: bad dtype %d", dtype);
  OES_REQUIRE(act == OES_ACT_NONE || act == OES_ACT_SWIGLU, "moe_fp8_quantize: bad act %d", act);
  if (T == 0) return OES_OK;
  OES_REQUIRE(x && q && scale, "moe_fp8_quantize: null pointer");
  OES_REQUIRE(x_ld >= (act == OES_ACT_SWIGLU ? 2 : 1) * (int64_t)K && q_ld >= K,
              "moe_fp8_quantize: a row stride is smaller than its row");
  OES_REQUIRE(((uintptr_t)x & (dtype == OES_BF16 ? 1 : 3)) == 0 && ((uintptr_t)scale & 3) == 0,
              "moe_fp8_quantize: a pointer is not aligned to its type");
  return fp8_quantize(x, dtype, x_ld, T, K, act, q, q_ld, scale, stream);
}
