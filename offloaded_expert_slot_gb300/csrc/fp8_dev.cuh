// 8-bit (e4m3) values with one fp32 scale for a group of 128: the quantiser
// shared by every kernel that writes them.
//
// For a group with amax = max |v| over its values that are not NaN, taken as
// at least 2^-100:
//   s = amax / 448,   code = e4m3(448 v / amax), the quotient rounded to fp32
// and then to the nearest code, ties to even.  448 is the largest e4m3 value,
// so the largest |v| of a group always gets the largest code.  The floor keeps
// an all-zero group free of divisions by zero (its codes are 0).  A NaN gets a
// NaN code; an infinity makes s infinite, so the whole group reads as NaN.
//
// The quotient is taken from the mathematics, four operations a value instead
// of a full division: with amax = m 2^e, m in [1, 2), and y = 1/m within 2^-23,
//   p = RN(v (7 2^(6-e))),  q0 = RN(p y),  q = RN(q0 + (p - q0 m) y)
// p - q0 m is exact in an FMA, so q = RN(p/m + d) with |d| below 2^-44 |q|
// (Markstein, IBM J. Res. Dev. 34, 1990): a quotient that is an fp32 number
// comes out exact.  That is what matters here: bf16 values reach exact
// midpoints between two codes all the time (448 v / amax is a ratio of small
// integers), and a midpoint off by one fp32 unit would round the wrong way.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace oes {

constexpr int kQuantGroup = 128;
constexpr float kCodeMax = 448.0f;

struct QuantScale {
  float s;         // what a code stands for: code * s
  float mul;       // 7 2^(6-e)
  float m, rcp_m;  // amax's significand and its reciprocal
};

__device__ __forceinline__ QuantScale quant_scale(float amax) {
  amax = fmaxf(amax, 0x1p-100f);
  QuantScale q;
  q.s = amax * (1.0f / kCodeMax);  // within 2 units of 2^-24 of the quotient
  const uint32_t b = __float_as_uint(amax);
  if (b == 0x7F800000u) {  // an infinity: finite values get 0, infinities NaN
    q.mul = 0.0f;
    q.m = q.rcp_m = 1.0f;
  } else {
    q.mul = 7.0f * __uint_as_float((260u - (b >> 23)) << 23);
    q.m = __uint_as_float((b & 0x007FFFFFu) | 0x3F800000u);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q.rcp_m) : "f"(q.m));
  }
  return q;
}

__device__ __forceinline__ float quant_ratio(float v, const QuantScale& q) {
  const float p = v * q.mul;
  const float q0 = p * q.rcp_m;
  return fmaf(fmaf(-q0, q.m, p), q.rcp_m, q0);
}

// two ratios -> two e4m3 codes (lo in the low byte), nearest even, saturating
__device__ __forceinline__ uint32_t cvt_f32x2_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t quant4(float a, float b, float c, float d, const QuantScale& q) {
  return cvt_f32x2_e4m3x2(quant_ratio(a, q), quant_ratio(b, q)) |
         (cvt_f32x2_e4m3x2(quant_ratio(c, q), quant_ratio(d, q)) << 16);
}
__device__ __forceinline__ uint8_t quant1(float a, const QuantScale& q) {
  return (uint8_t)(cvt_f32x2_e4m3x2(quant_ratio(a, q), 0.0f) & 0xFFu);
}

// ----- rows of bf16 or fp32, read and written VEC values at a time
__device__ __forceinline__ float bf16_f32(uint32_t bits) { return __uint_as_float(bits << 16); }
__device__ __forceinline__ uint32_t f32_bf16(float v) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}
// two values -> bf16x2, lo in the low half
__device__ __forceinline__ uint32_t f32x2_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int VEC>
__device__ __forceinline__ void load_vals(const uint16_t* p, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_f32(u[i] & 0xFFFFu);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = bf16_f32(p[i]);
  }
}
template <int VEC>
__device__ __forceinline__ void load_vals(const float* p, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = p[i];
  }
}
template <int VEC>
__device__ __forceinline__ void store_vals(uint16_t* p, const float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = f32x2_bf16x2(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) p[i] = (uint16_t)f32_bf16(v[i]);
  }
}
template <int VEC>
__device__ __forceinline__ void store_vals(float* p, const float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) p[i] = v[i];
  }
}

__device__ __forceinline__ float sigmoid_f32(float g) { return 1.0f / (1.0f + expf(-g)); }

// g / (1 + exp(-g)) where it runs beside MMAs or loads: two special-function
// operations and eight others.  With e = exp(g) it is g e / (1 + e), and e enters
// as the product of two factors z = exp(g / 2), the second one only after g, so
// that nothing overflows or is flushed on the way: exp(-g) itself overflows
// below g = -88.7, and its reciprocal is flushed from -87.3 (with it, 4096 tokens x
// 10 took 491 us, like this 498).  z = 2^t with t = g log2(e) / 2 rounded, and e =
// z^2 (1 + lo), lo = g - 2 t ln 2 being what the rounding left.  From g = 64 ln 2 on
// the factor of g is exactly 1.  -inf gives NaN, like the quotient.  Within 17
// units of 2^-24 (measured: 8), a subnormal result rounded once more.
__device__ __forceinline__ float silu_f32(float g) {
  constexpr float kHalfLog2e = 0.721347511f, kTwoLn2 = 1.386294365f, kMost = 44.3614197f;
  const float c = fminf(g, kMost), t = c * kHalfLog2e;
  float z, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(z) : "f"(t));
  const float w = fmaf(z, fmaf(t, -kTwoLn2, c), z);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(w, z, 1.0f)));
  return w * r * g * z;
}

}  // namespace oes
