// moe_int8_quantize: rows of bf16 or fp32, or SwiGLU of such rows, to 8-bit
// integers with one fp32 scale a row.
//
//   amax = max |v| over the row, at least 2^-100,   scale = amax / 127,
//   code = the integer nearest to 127 v / amax, ties to even
//
// The quotient that decides is the real number, not a rounded one.  In fp32,
// f = v (127 / amax) is within 2^-16 of it (|f| <= 127, two roundings), which
// settles every code but those of an f that close to m + 1/2.  There 254 |v| is
// compared with (2 m + 1) amax, both as the sum of an fp32 product and what it left
// (an FMA): the products are so close that their difference is exact, and the sign of
// the sum of both differences is right.  bf16 rows meet such ties often (any amax with
// a factor of 127), and a tie decided by a rounded quotient would go either
// way.  (In 64 bits the comparison is shorter, but GB300's rate for them is so low that
// 4096 x 2048 took 25 us.)  The floor on amax keeps rows of zeros and of the smallest
// numbers free of infinite factors (their codes are 0).  A row with a NaN or an
// infinity gets a NaN scale and zeros.
//
// Bound by memory traffic (3 bytes a value from bf16): the row is held in
// registers between the maximum and the codes, up to 32 values a thread; what is
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

// What a row's codes are made with.
struct RowScale {
  float rcp;        // 127 / amax
  float unit, top;  // a power of two, and amax times it, in [2, 4)
};

// The code's size where |f| is next to m + 1/2: m or m + 1.
__device__ __forceinline__ uint32_t int8_next_to_tie(float v, const RowScale& rs) {
  const float m = floorf(fabsf(v) * rs.rcp), odd = 2.0f * m + 1.0f, a = fabsf(v) * rs.unit;
  const float l = 254.0f * a, r = odd * rs.top;
  const float past = (l - r) + (fmaf(254.0f, a, -l) - fmaf(odd, rs.top, -r));
  const uint32_t c = (uint32_t)m;
  return c + (past > 0.0f || (past == 0.0f && (c & 1u)) ? 1u : 0u);
}

// V codes, one in each low byte.  Adding 3 2^22 leaves the nearest integer of v rcp
// (an FMA: the product unrounded) in the low bits of the sum, in two's complement;
// d is how far it is from there.
template <int V>
__device__ __forceinline__ void int8_codes(const float (&v)[V], const RowScale& rs, uint32_t (&code)[V]) {
  constexpr float kMagic = 12582912.0f, kNear = 0.5f - 0x1p-14f;
  float d[V], far = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float t = fmaf(v[i], rs.rcp, kMagic);
    d[i] = fabsf(fmaf(v[i], rs.rcp, -(t - kMagic)));
    far = fmaxf(far, d[i]);
    code[i] = __float_as_uint(t);
  }
  if (far > kNear) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (d[i] > kNear) {
        const uint32_t c = int8_next_to_tie(v[i], rs);
        code[i] = v[i] < 0.0f ? 0u - c : c;
      }
  }
}

// A thread's V values of a chunk, held between the maximum and the codes: bf16 rows as
// they come, half the registers of fp32.
template <int V, bool SWIGLU, typename XT>
struct Chunk {
  static constexpr bool kRaw = V == 8 && !SWIGLU && sizeof(XT) == 2;
  uint4 raw;
  float v[kRaw ? 1 : V];
  __device__ __forceinline__ void load(const XT* x, int c, int K, bool in) {
    if constexpr (kRaw) {
      raw = make_uint4(0u, 0u, 0u, 0u);
      if (in) raw = *reinterpret_cast<const uint4*>(x + (int64_t)c * V);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = 0.0f;
      if (!in) return;
      load_vals<V>(x + (int64_t)c * V, v);
      if (SWIGLU) {
        float u[V];
        load_vals<V>(x + K + (int64_t)c * V, u);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = silu_f32(v[i]) * u[i];
      }
    }
  }
  // sizes order like their bits, with infinities and NaN on top
  __device__ __forceinline__ uint32_t most(uint32_t m) const {
    if constexpr (kRaw) {
      const uint32_t a = __vmaxu2(__vmaxu2(raw.x & 0x7FFF7FFFu, raw.y & 0x7FFF7FFFu),
                                  __vmaxu2(raw.z & 0x7FFF7FFFu, raw.w & 0x7FFF7FFFu));
      return max(m, max(a << 16, a & 0xFFFF0000u));
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
      return m;
    }
  }
  __device__ __forceinline__ void store(int8_t* q, int c, const RowScale& rs, bool odd) const {
    float w[V];
    if constexpr (kRaw) {
      const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[2 * i] = bf16_f32(u[i] & 0xFFFFu);
        w[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = v[i];
    }
    uint32_t code[V];
    int8_codes<V>(w, rs, code);
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
  }
};

// V values a load (8, or 1 where rows are not aligned for it), TPR threads a row,
// the first H chunks of each thread held.
template <int V, bool SWIGLU, typename XT, int TPR, int H>
__global__ void __launch_bounds__(256) int8_quantize_kernel(const Int8QuantArgs a) {
  pdl_begin();
  constexpr int kRows = 256 / TPR;  // rows a CTA
  constexpr int kW = TPR / 32;      // warps a row
  __shared__ uint32_t s_max[kRows][kW];
  const int tid = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int nc = a.K / V;
  for (int64_t t0 = (int64_t)blockIdx.x * kRows; t0 < a.T; t0 += (int64_t)gridDim.x * kRows) {
    const int64_t t = t0 + sub;
    const bool live = t < a.T;
    const XT* x = static_cast<const XT*>(a.x) + (live ? t : 0) * a.ld;
    Chunk<V, SWIGLU, XT> held[H];
    uint32_t m = 0;
    if (live) {
#pragma unroll
      for (int h = 0; h < H; ++h) held[h].load(x, tid + h * TPR, a.K, tid + h * TPR < nc);
#pragma unroll
      for (int h = 0; h < H; ++h) m = held[h].most(m);
      for (int c = tid + H * TPR; c < nc; c += TPR) {
        Chunk<V, SWIGLU, XT> w;
        w.load(x, c, a.K, true);
        m = w.most(m);
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
    const float amax = fmaxf(__uint_as_float(odd ? 0u : m), 0x1p-100f);
    RowScale rs;
    rs.rcp = odd ? 0.0f : __fdiv_rn(127.0f, amax);
    rs.unit = __uint_as_float((255u - (__float_as_uint(amax) >> 23)) << 23);
    rs.top = amax * rs.unit;
    if (tid == 0) a.s[t] = odd ? __int_as_float(0x7FFFFFFF) : __fdiv_rn(amax, 127.0f);
    int8_t* q = a.q + t * a.q_ld;
#pragma unroll
    for (int h = 0; h < H; ++h)
      if (tid + h * TPR < nc) held[h].store(q, tid + h * TPR, rs, odd);
    for (int c = tid + H * TPR; c < nc; c += TPR) {
      Chunk<V, SWIGLU, XT> w;
      w.load(x, c, a.K, true);
      w.store(q, c, rs, odd);
    }
  }
}

template <int V, bool SWIGLU, typename XT, int TPR, int H>
int launch_rows(const Int8QuantArgs& a, cudaStream_t stream) {
  const int64_t ctas = ceil_div64(a.T, 256 / TPR);
  launch_kernel(int8_quantize_kernel<V, SWIGLU, XT, TPR, H>, (int)std::min<int64_t>(ctas, (int64_t)num_sms() * 8),
                256, 0, stream, a);
  OES_CHECK_LAUNCH("int8_quantize_kernel");
  return OES_OK;
}

// Threads a row: a CTA where there are few rows or they are long, else as few as hold
// the row in two to four chunks each.  4096 x 2048 bf16: 6.3 us with 128 threads a row
// (4.0 TB/s), 6.6 with 64, 8.4 with 32, 7.2 with 256; 8192 x 256 4.9, 5.7, 8.0 and 10.4
// with 32, 64, 128 and 256; 16384 x 4096 37.7 with 128 of four chunks, 42 to 59 with
// others; 600 x 2048 2.4 with 256 and 6.0 with 32.
template <int V, bool SWIGLU, typename XT>
int launch_int8_quant(const Int8QuantArgs& a, cudaStream_t stream) {
  const int nc = a.K / V;
  const bool many = a.T >= 4 * num_sms();
  if constexpr (V == 8) {
    if (many && nc <= 64) return launch_rows<V, SWIGLU, XT, 32, 2>(a, stream);
    if (many && nc <= 128) return launch_rows<V, SWIGLU, XT, 64, 2>(a, stream);
    if (many && nc <= 256) return launch_rows<V, SWIGLU, XT, 128, 2>(a, stream);
    if (many && nc <= 512) return launch_rows<V, SWIGLU, XT, 128, 4>(a, stream);
    if (nc <= 256) return launch_rows<V, SWIGLU, XT, 256, 1>(a, stream);
    return launch_rows<V, SWIGLU, XT, 256, 4>(a, stream);
  } else {
    if (many && nc <= 1024) return launch_rows<V, SWIGLU, XT, 32, 32>(a, stream);
    return launch_rows<V, SWIGLU, XT, 256, 16>(a, stream);
  }
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
