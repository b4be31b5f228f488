// moe_block_norm: the residual update after a block and the norm before the
// next one, in one pass over the rows.
//
//   v  = y * rsqrt(mean(y^2) + eps) * (offset + w_post)       (or v = y)
//   r' = residual + residual_scale * gate * v
//   u  = r' * rsqrt(mean(r'^2) + eps) * (offset + w_pre)      (or u = r')
//
// Every sum and product is fp32; r' goes into the second norm unrounded, and
// the codes are taken from the unrounded u, so each output is rounded once.
// What bounds it is memory traffic: 8 bytes a value in bf16 (9 with codes)
// against about a dozen operations.  So a row is read once, kept in registers
// across both reductions, and written once.  4096 x 2048 with both norms, a
// gate a token and codes takes 16.0 us, 4.7 TB/s; a row takes a CTA of 128
// threads with 16 values each, where a warp a row took 45 us, 64 threads 29 and
// 256 threads 25.
#include <algorithm>

#include "common.cuh"
#include "fp8_dev.cuh"
#include "internal.h"

namespace oes {
namespace {

constexpr int kMaxH = 16384;
constexpr int kNormResident = 512;  // threads an SM holds at once

// CTAs an SM shall hold, 0 to leave that to the compiler: rows of single values
// are short of loads in flight, so their threads get 64 registers at most.
constexpr int norm_ctas(int vec, int maxt) { return vec == 1 && maxt <= 512 ? 2 : 0; }

// VEC values of a row as they lie in memory.
template <int VEC, typename T>
struct Raw {
  T v[VEC];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC == 8) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(v)[i] = reinterpret_cast<const uint4*>(p)[i];
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = p[i];
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 2) return bf16_f32(v[i]);
    else return v[i];
  }
};

// RT: uint16_t (bf16) or float residual.  Value e of chunk j of a row belongs
// to thread (j * threads + tid) as value VEC * that + e.  WARP: a warp a row,
// else a CTA a row.  GATED: the gate has a value a channel or an element.  A
// CTA walks rows; where registers allow (kAhead) its weights stay in them and
// the next row is on its way while this one is reduced.
template <int VEC, int NV, bool WARP, int MAXT, bool GATED, typename RT>
__global__ void __launch_bounds__(MAXT, norm_ctas(VEC, MAXT)) block_norm_kernel(const oes_block_norm p) {
  pdl_begin();
  constexpr bool kAhead = VEC == 8 && MAXT <= 512;
  __shared__ float red[2][32];
  __shared__ float gmax[VEC == 1 ? NV : 1][32];
  __shared__ QuantScale gscale[VEC == 1 ? NV : 1][8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nthr = WARP ? 32 : blockDim.x;
  const int tid = WARP ? lane : threadIdx.x;
  const int nw = blockDim.x >> 5;
  const int64_t step = (int64_t)gridDim.x * (WARP ? nw : 1);
  const float inv_h = 1.0f / (float)p.H;
  // The two buffers take turns: a warp writes one again only past the barrier of
  // the sum between, which every warp reaches after it has read the first.
  int turn = 0;
  auto row_sum = [&](float s) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (WARP) return s;
    float* sums = red[turn];
    turn ^= 1;
    if (lane == 0) sums[warp] = s;
    __syncthreads();
    s = lane < nw ? sums[lane] : 0.0f;
#pragma unroll
    for (int o = MAXT / 64; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return __shfl_sync(0xffffffffu, s, 0);
  };
  auto col = [&](int j) { return (j * nthr + tid) * VEC; };
  using W = Raw<VEC, uint16_t>;
  auto load_w = [&](const uint16_t* w, int j) {
    W x = {};
    if (w && col(j) < p.H) x.load(w + col(j));
    return x;
  };
  W wpost[NV], wpre[NV];
  if (kAhead) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      wpost[j] = load_w(p.post_weight, j);
      wpre[j] = load_w(p.pre_weight, j);
    }
  }
  Raw<VEC, RT> rn[NV] = {};
  W yn[NV] = {};
  float gn = 0.0f;
  auto fetch = [&](int64_t row) {
    if (row >= p.T) return;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (col(j) >= p.H) continue;
      rn[j].load(static_cast<const RT*>(p.residual) + row * p.residual_ld + col(j));
      if (p.y) yn[j].load(p.y + row * p.y_ld + col(j));
    }
    if (p.gate_kind == OES_GATE_TOKEN) gn = static_cast<const float*>(p.gate)[row * p.gate_ld];
  };
  int64_t row = WARP ? (int64_t)blockIdx.x * nw + warp : blockIdx.x;
  if (kAhead) fetch(row);
  for (; row < p.T; row += step) {
    float r[NV][VEC];
    float v[NV][VEC];
    if (!kAhead) fetch(row);
    const float gt = gn;
    W ge[GATED ? NV : 1];
    if (GATED) {
      const uint16_t* g = static_cast<const uint16_t*>(p.gate) + (p.gate_kind == OES_GATE_ELEMENT ? row * p.gate_ld : 0);
#pragma unroll
      for (int j = 0; j < NV; ++j) ge[j] = load_w(g, j);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        r[j][e] = col(j) < p.H ? rn[j].at(e) : 0.0f;
        v[j][e] = p.y && col(j) < p.H ? yn[j].at(e) : 0.0f;
      }
    if (kAhead) fetch(row + step);
    float s = 0.0f;
    if (p.y) {
      float k = p.residual_scale;
      if (p.gate_kind == OES_GATE_TOKEN) k *= p.gate_sigmoid ? sigmoid_f32(gt) : gt;
      float inv = 1.0f;
      if (p.post_weight) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int e = 0; e < VEC; ++e) s = fmaf(v[j][e], v[j][e], s);
        inv = rsqrtf(row_sum(s) * inv_h + p.eps);
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (col(j) >= p.H) continue;
        const W w = kAhead ? wpost[j] : load_w(p.post_weight, j);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          if (p.post_weight) v[j][e] = v[j][e] * inv * (p.weight_offset + w.at(e));
          if (GATED) {
            const float g = ge[j].at(e);
            v[j][e] *= p.gate_sigmoid ? sigmoid_f32(g) : g;
          }
          r[j][e] = fmaf(k, v[j][e], r[j][e]);
        }
      }
    }
    if (p.out_residual) {
      RT* op = static_cast<RT*>(p.out_residual) + row * p.out_residual_ld;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (col(j) < p.H) store_vals<VEC>(op + col(j), r[j]);
    }
    if (!p.out && !p.out_q) continue;
    if (p.pre_weight) {
      s = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) s = fmaf(r[j][e], r[j][e], s);
      const float inv = rsqrtf(row_sum(s) * inv_h + p.eps);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (col(j) >= p.H) continue;
        const W w = kAhead ? wpre[j] : load_w(p.pre_weight, j);
#pragma unroll
        for (int e = 0; e < VEC; ++e) r[j][e] = r[j][e] * inv * (p.weight_offset + w.at(e));
      }
    }
    if (p.out) {
      uint16_t* op = p.out + row * p.out_ld;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (col(j) < p.H) store_vals<VEC>(op + col(j), r[j]);
    }
    if (p.out_q) {
      uint8_t* qp = p.out_q + row * p.out_q_ld;
      float* sp = p.out_scale + row * ((p.H + kQuantGroup - 1) / kQuantGroup);
      float a[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        a[j] = 0.0f;  // values past H are 0
#pragma unroll
        for (int e = 0; e < VEC; ++e) a[j] = fmaxf(a[j], fabsf(r[j][e]));
        // a group is 16 neighbouring lanes of 8 values, or four warps of one
#pragma unroll
        for (int o = VEC == 8 ? 8 : 16; o >= 1; o >>= 1)
          a[j] = fmaxf(a[j], __shfl_xor_sync(0xffffffffu, a[j], o));
        if (VEC == 1 && lane == 0) gmax[j][warp] = a[j];
      }
      if (VEC == 1) {
        // a group's scale is worked out once, by one of its four warps
        __syncthreads();
        if ((warp & 3) == 0 && lane < NV) {
          const float* g = gmax[lane] + warp;
          gscale[lane][warp >> 2] = quant_scale(fmaxf(fmaxf(g[0], g[1]), fmaxf(g[2], g[3])));
        }
        __syncthreads();
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = col(j);
        if (c >= p.H) continue;
        const QuantScale qs = VEC == 8 ? quant_scale(a[j]) : gscale[VEC == 8 ? 0 : j][warp >> 2];
        if constexpr (VEC == 8) {
          *reinterpret_cast<uint2*>(qp + c) =
              make_uint2(quant4(r[j][0], r[j][1], r[j][2], r[j][3], qs),
                         quant4(r[j][4], r[j][5], r[j][6], r[j][7], qs));
        } else {
          qp[c] = quant1(r[j][0], qs);
        }
        if (c % kQuantGroup == 0) sp[c / kQuantGroup] = qs.s;
      }
      if (VEC == 1) __syncthreads();  // gmax is read before the next row's is written
    }
  }
}

template <int VEC, int NV, bool WARP, int MAXT>
int launch_norm(const oes_block_norm& p, int threads, cudaStream_t stream) {
  const int rows = WARP ? threads / 32 : 1;
  const int64_t want = ceil_div64(p.T, rows);
  // about the CTAs that are resident at once, so that each walks its rows
  const int grid =
      (int)std::min<int64_t>(want, (int64_t)num_sms() * std::max(1, (VEC == 8 ? kNormResident : 2048) / threads));
  auto go = [&](auto kernel) { launch_kernel(kernel, grid, threads, 0, stream, p); };
  const bool gated = p.gate_kind >= OES_GATE_CHANNEL;
  if (p.dtype == OES_BF16) {
    if (gated) go(block_norm_kernel<VEC, NV, WARP, MAXT, true, uint16_t>);
    else go(block_norm_kernel<VEC, NV, WARP, MAXT, false, uint16_t>);
  } else {
    if (gated) go(block_norm_kernel<VEC, NV, WARP, MAXT, true, float>);
    else go(block_norm_kernel<VEC, NV, WARP, MAXT, false, float>);
  }
  OES_CHECK_LAUNCH("block_norm_kernel");
  return OES_OK;
}

}  // namespace
}  // namespace oes

using namespace oes;

extern "C" int moe_block_norm(const oes_block_norm* a, oes_stream_t stream) {
  OES_REQUIRE(a, "moe_block_norm: null arguments");
  const oes_block_norm& p = *a;
  OES_REQUIRE(p.T >= 0 && p.H >= 1, "moe_block_norm: bad T=%d H=%d", p.T, p.H);
  if (p.H > kMaxH) {
    set_error("moe_block_norm: H=%d is over %d", p.H, kMaxH);
    return OES_ERR_UNSUPPORTED;
  }
  OES_REQUIRE(p.dtype == OES_BF16 || p.dtype == OES_F32, "moe_block_norm: bad dtype %d", p.dtype);
  OES_REQUIRE(p.gate_kind >= OES_GATE_NONE && p.gate_kind <= OES_GATE_ELEMENT,
              "moe_block_norm: bad gate_kind %d", p.gate_kind);
  OES_REQUIRE(p.eps >= 0.0f, "moe_block_norm: eps must not be negative");
  OES_REQUIRE(p.out_residual || p.out || p.out_q, "moe_block_norm: no output");
  OES_REQUIRE((p.out_q == nullptr) == (p.out_scale == nullptr),
              "moe_block_norm: out_q and out_scale go together");
  OES_REQUIRE(p.y || (!p.post_weight && p.gate_kind == OES_GATE_NONE),
              "moe_block_norm: post_weight and gate need y");
  OES_REQUIRE((p.gate != nullptr) == (p.gate_kind != OES_GATE_NONE),
              "moe_block_norm: gate and gate_kind disagree");
  if (p.T == 0) return OES_OK;
  OES_REQUIRE(p.residual, "moe_block_norm: null residual");
  const bool elem = p.gate_kind == OES_GATE_ELEMENT;
  OES_REQUIRE(p.residual_ld >= p.H && (!p.y || p.y_ld >= p.H) && (!elem || p.gate_ld >= p.H) &&
                  (p.gate_kind != OES_GATE_TOKEN || p.gate_ld >= 1) &&
                  (!p.out_residual || p.out_residual_ld >= p.H) && (!p.out || p.out_ld >= p.H) &&
                  (!p.out_q || p.out_q_ld >= p.H),
              "moe_block_norm: a row stride is smaller than its row");
  const uintptr_t ra = p.dtype == OES_BF16 ? 2 : 4;
  auto at = [](const void* q, uintptr_t n) { return ((uintptr_t)q & (n - 1)) == 0; };
  OES_REQUIRE(at(p.residual, ra) && at(p.out_residual, ra) && at(p.y, 2) && at(p.post_weight, 2) &&
                  at(p.pre_weight, 2) && at(p.gate, p.gate_kind == OES_GATE_TOKEN ? 4 : 2) &&
                  at(p.out, 2) && at(p.out_scale, 4),
              "moe_block_norm: a pointer is not aligned to its type");
  // rows of 8 values a load when every row and weight is aligned for it
  const int64_t rm = 16 / (int64_t)ra;
  const bool vec = p.H % 8 == 0 && at(p.residual, 16) && p.residual_ld % rm == 0 &&
                   (!p.y || (at(p.y, 16) && p.y_ld % 8 == 0)) && at(p.post_weight, 16) &&
                   at(p.pre_weight, 16) && (p.gate_kind < OES_GATE_CHANNEL || at(p.gate, 16)) &&
                   (!elem || p.gate_ld % 8 == 0) &&
                   (!p.out_residual || (at(p.out_residual, 16) && p.out_residual_ld % rm == 0)) &&
                   (!p.out || (at(p.out, 16) && p.out_ld % 8 == 0)) &&
                   (!p.out_q || (at(p.out_q, 8) && p.out_q_ld % 8 == 0));
  auto up = [](int n, int m) { return (n + m - 1) / m * m; };
  if (vec) {
    const int c = p.H / 8, half = up(ceil_div(c, 2), 32);  // 16 values a thread
    if (c <= 64) return launch_norm<8, 2, true, 128>(p, 128, stream);
    if (half <= 128) return launch_norm<8, 2, false, 128>(p, half, stream);
    if (half <= 256) return launch_norm<8, 2, false, 256>(p, half, stream);
    if (half <= 512) return launch_norm<8, 2, false, 512>(p, half, stream);
    return launch_norm<8, 2, false, 1024>(p, half, stream);
  }
  if (p.H <= 2048) return launch_norm<1, 4, false, 512>(p, up(ceil_div(p.H, 4), 128), stream);
  if (p.H <= 4096) return launch_norm<1, 4, false, 1024>(p, up(ceil_div(p.H, 4), 128), stream);
  return launch_norm<1, 16, false, 1024>(p, up(ceil_div(p.H, 16), 128), stream);
}
