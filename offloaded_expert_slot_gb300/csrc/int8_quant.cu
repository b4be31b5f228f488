// moe_int8_quantize: rows of bf16 or fp32, or SwiGLU of such rows, to 8-bit
// integers with one fp32 scale a row.
//
//   amax = max |v| over the row, at least 2^-100,   scale = amax / 127,
//   code = the integer nearest to 127 v / amax, ties to even
//
// The quotient that decides is the real number, not a rounded one.  In fp32,
// f = v (127 / amax) is within 2^-16 of it (|f| <= 127, two roundings), which
// settles every code but those of an f that close to m + 1/2.  There the exact
// comparison 254 |v| against (2 m + 1) amax is made, in 64 bits, where both
// sides are exact (24 + 8 bits).  bf16 rows meet such ties often (any amax with
// a factor of 127), and a tie decided by a rounded quotient would go either
// way.  The floor on amax keeps rows of zeros and of the smallest numbers free
// of infinite factors (their codes are 0).  A row with a NaN or an infinity gets
// a NaN scale and zeros.
//
// Bound by memory traffic (3 bytes a value from bf16): the row is held in
// registers between the maximum and the codes, up to 64 values a thread; what is
// past that is read again.
#include <algorithm>

#include "common.cuh"
#include "fp8_dev.cuh"

namespace oes {
namespace {

struct Int8QuantArgs {
  const void* x;
  int64_t ld;  // of x, in values
  int T, K;
  int8_t* q;
  int64_t q_ld;
  float* s;
};

// The code of one value, exactly: m or m + 1, m = floor(|f|).  Out of line, since
// one chunk in a thousand comes here.
__device__ __noinline__ int int8_code_exact(float v, float rcp, float amax) {
  const float a = fabsf(v), m = floorf(a * rcp);
  const double lhs = 254.0 * (double)a, rhs = (2.0 * (double)m + 1.0) * (double)amax;
  int c = (int)m;
  if (lhs > rhs || (lhs == rhs && (c & 1))) ++c;
  return v < 0.0f ? -c : c;
}

// V codes, one in each low byte.  Adding 3 2^22 leaves the nearest integer of v rcp
// (an FMA: the product unrounded) in the low bits of the sum, in two's complement;
// d is how far it is from there.
template <int V>
__device__ __forceinline__ void int8_codes(const float (&v)[V], float rcp, float amax, uint32_t (&code)[V]) {
  constexpr float kMagic = 12582912.0f;
  float far = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float t = fmaf(v[i], rcp, kMagic);
    far = fmaxf(far, fabsf(fmaf(v[i], rcp, -(t - kMagic))));
    code[i] = __float_as_uint(t);
  }
  if (far > 0.5f - 0x1p-14f) {
#pragma unroll
    for (int i = 0; i < V; ++i) code[i] = (uint32_t)int8_code_exact(v[i], rcp, amax);
  }
}

// The values of chunk c of a row (V at a time), K past its end as zeros.
template <int V, bool SWIGLU, typename XT>
__device__ __forceinline__ void chunk_vals(const XT* x, int c, int K, float (&v)[V]) {
  load_vals<V>(x + (int64_t)c * V, v);
  if (SWIGLU) {
    float u[V];
    load_vals<V>(x + K + (int64_t)c * V, u);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = silu_f32(v[i]) * u[i];
  }
}

// V values a load (8, or 1 where rows are not aligned for it), TPR threads a row,
// the first H chunks of each thread held.
template <int V, bool SWIGLU, typename XT, int TPR, int H>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) int8_quantize_kernel(const Int8QuantArgs a) {
  pdl_begin();
  constexpr int kRows = TPR < 256 ? 256 / TPR : 1;  // rows a CTA
  constexpr int kW = TPR / 32;                       // warps a row
  __shared__ uint32_t s_max[kRows][kW];
  const int tid = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int nc = a.K / V;
  for (int64_t t0 = (int64_t)blockIdx.x * kRows; t0 < a.T; t0 += (int64_t)gridDim.x * kRows) {
    const int64_t t = t0 + sub;
    const bool live = t < a.T;
    const XT* x = static_cast<const XT*>(a.x) + (live ? t : 0) * a.ld;
    float v[H][V];
    uint32_t m = 0;  // sizes order like their bits, with infinities and NaN on top
    if (live) {
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const int c = tid + h * TPR;
        if (c < nc) {
          chunk_vals<V, SWIGLU>(x, c, a.K, v[h]);
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) v[h][i] = 0.0f;
        }
      }
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int i = 0; i < V; ++i) m = max(m, __float_as_uint(v[h][i]) & 0x7FFFFFFFu);
      for (int c = tid + H * TPR; c < nc; c += TPR) {
        float w[V];
        chunk_vals<V, SWIGLU>(x, c, a.K, w);
#pragma unroll
        for (int i = 0; i < V; ++i) m = max(m, __float_as_uint(w[i]) & 0x7FFFFFFFu);
      }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (kW > 1) {
      if ((tid & 31) == 0) s_max[sub][tid >> 5] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kW; ++w) m = max(m, s_max[sub][w]);
      __syncthreads();  // the next row's maxima go to the same place
    }
    if (!live) continue;
    const bool odd = m >= 0x7F800000u;
    const float amax = fmaxf(__uint_as_float(m), 0x1p-100f);
    const float rcp = odd ? 0.0f : __fdiv_rn(127.0f, amax);
    if (tid == 0) a.s[t] = odd ? __int_as_float(0x7FFFFFFF) : __fdiv_rn(amax, 127.0f);
    int8_t* q = a.q + t * a.q_ld;
    auto put = [&](int c, float (&w)[V]) {
      uint32_t code[V];
      int8_codes<V>(w, rcp, amax, code);
      if (odd) {
#pragma unroll
        for (int i = 0; i < V; ++i) code[i] = 0u;
      }
      if constexpr (V == 8) {
        uint32_t o[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
          o[j] = __byte_perm(__byte_perm(code[4 * j], code[4 * j + 1], 0x0040),
                             __byte_perm(code[4 * j + 2], code[4 * j + 3], 0x0040), 0x5410);
        *reinterpret_cast<uint2*>(q + (int64_t)c * 8) = make_uint2(o[0], o[1]);
      } else {
        q[c] = (int8_t)code[0];
      }
    };
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int c = tid + h * TPR;
      if (c < nc) put(c, v[h]);
    }
    for (int c = tid + H * TPR; c < nc; c += TPR) {
      float w[V];
      chunk_vals<V, SWIGLU>(x, c, a.K, w);
      put(c, w);
    }
  }
}

template <int V, bool SWIGLU, typename XT, int TPR, int H>
int launch_rows(const Int8QuantArgs& a, cudaStream_t stream) {
  constexpr int threads = TPR < 256 ? 256 : TPR;
  const int64_t ctas = ceil_div64(a.T, threads / TPR);
  launch_kernel(int8_quantize_kernel<V, SWIGLU, XT, TPR, H>, (int)std::min<int64_t>(ctas, (int64_t)num_sms() * 8),
                threads, 0, stream, a);
  OES_CHECK_LAUNCH("int8_quantize_kernel");
  return OES_OK;
}

// A warp a row where there are rows for all SMs and it holds them, else a CTA.
template <int V, bool SWIGLU, typename XT>
int launch_int8_quant(const Int8QuantArgs& a, cudaStream_t stream) {
  constexpr int H = V == 8 ? 8 : 32;
  if (a.K <= 32 * H * V && a.T >= num_sms() * 4) return launch_rows<V, SWIGLU, XT, 32, H>(a, stream);
  return launch_rows<V, SWIGLU, XT, 256, V == 8 ? 4 : 16>(a, stream);
}

template <int V>
int launch_int8_quant_of(const Int8QuantArgs& a, int dtype, int act, cudaStream_t stream) {
  if (act == OES_ACT_SWIGLU)
    return dtype == OES_BF16 ? launch_int8_quant<V, true, uint16_t>(a, stream)
                             : launch_int8_quant<V, true, float>(a, stream);
  return dtype == OES_BF16 ? launch_int8_quant<V, false, uint16_t>(a, stream)
                           : launch_int8_quant<V, false, float>(a, stream);
}

}  // namespace
}  // namespace oes

using namespace oes;

extern "C" int moe_int8_quantize(const void* x, int dtype, int64_t x_ld, int T, int K, int act, int8_t* q,
                                 int64_t q_ld, float* scale, oes_stream_t stream) {
  OES_REQUIRE(T >= 0 && K >= 1 && K <= (1 << 28), "moe_int8_quantize: bad T=%d K=%d", T, K);
  OES_REQUIRE(dtype == OES_BF16 || dtype == OES_F32, "moe_int8_quantize: bad dtype %d", dtype);
  OES_REQUIRE(act == OES_ACT_NONE || act == OES_ACT_SWIGLU, "moe_int8_quantize: bad act %d", act);
  if (T == 0) return OES_OK;
  OES_REQUIRE(x && q && scale, "moe_int8_quantize: null pointer");
  OES_REQUIRE(x_ld >= (act == OES_ACT_SWIGLU ? 2 : 1) * (int64_t)K && q_ld >= K,
              "moe_int8_quantize: a row stride is smaller than its row");
  OES_REQUIRE(((uintptr_t)x & (dtype == OES_BF16 ? 1 : 3)) == 0 && ((uintptr_t)scale & 3) == 0,
              "moe_int8_quantize: a pointer is not aligned to its type");
  Int8QuantArgs a{x, x_ld, T, K, q, q_ld, scale};
  // eight values a load where rows, both halves and codes are aligned for it
  const int64_t m = dtype == OES_BF16 ? 8 : 4;
  const bool vec = K % 8 == 0 && ((uintptr_t)x & 15) == 0 && x_ld % m == 0 && ((uintptr_t)q & 7) == 0 && q_ld % 8 == 0;
  return vec ? launch_int8_quant_of<8>(a, dtype, act, stream) : launch_int8_quant_of<1>(a, dtype, act, stream);
}
