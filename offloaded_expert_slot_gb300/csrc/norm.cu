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
// across both reductions, and written once.  In rows of 16-byte loads, 4096 x
// 2048 with both norms, a gate a token and codes takes 16.0 us, 4.7 TB/s; a row
// takes a CTA of 128 threads with 16 values each, where a warp a row took 45 us,
// 64 threads 29 and 256 threads 25.
#include <algorithm>

#include "common.cuh"
#include "fp8_dev.cuh"
#include "internal.h"

namespace oes {
namespace {

constexpr int kMaxH = 16384;
constexpr int kNormResident = 512;  // threads an SM holds at once
constexpr int kAnyResident = 1024;  // the same for block_norm_any_kernel
constexpr int kAnySmem = 216 << 10;  // of an SM, for its CTAs' rows

// The sum of a value over the threads of a row: a warp, or the nw warps of a
// CTA (at most MAXT / 32).  The two buffers take turns: a warp writes one again
// only past the barrier of the sum between, which every warp reaches after it
// has read the first.
template <bool WARP, int MAXT>
struct RowSum {
  float (*bufs)[32];
  int nw, turn;
  __device__ __forceinline__ float operator()(float s) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (WARP) return s;
    const int lane = threadIdx.x & 31;
    float* sums = bufs[turn];
    turn ^= 1;
    if (lane == 0) sums[threadIdx.x >> 5] = s;
    __syncthreads();
    s = lane < nw ? sums[lane] : 0.0f;
#pragma unroll
    for (int o = MAXT / 64; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return __shfl_sync(0xffffffffu, s, 0);
  }
};

__device__ __forceinline__ float widen(uint16_t v) { return bf16_f32(v); }
__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ void narrow(uint16_t* p, float v) { *p = (uint16_t)f32_bf16(v); }
__device__ __forceinline__ void narrow(float* p, float v) { *p = v; }

// ------------------------------------------------- rows of 16-byte loads
// 8 values of a row as they lie in memory.
template <typename T>
struct Raw {
  T v[8];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(v)[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ float at(int i) const { return widen(v[i]); }
};

// RT: uint16_t (bf16) or float residual.  Value e of chunk j of a row belongs
// to thread (j * threads + tid) as value 8 * that + e.  WARP: a warp a row,
// else a CTA a row.  GATED: the gate has a value a channel or an element.  A
// CTA walks rows; where registers allow (kAhead) its weights stay in them and
// the next row is on its way while this one is reduced.
template <int NV, bool WARP, int MAXT, bool GATED, typename RT>
__global__ void __launch_bounds__(MAXT) block_norm_kernel(const oes_block_norm p) {
  pdl_begin();
  constexpr bool kAhead = MAXT <= 512;
  __shared__ float red[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nthr = WARP ? 32 : blockDim.x;
  const int tid = WARP ? lane : threadIdx.x;
  const int nw = blockDim.x >> 5;
  const int64_t step = (int64_t)gridDim.x * (WARP ? nw : 1);
  const float inv_h = 1.0f / (float)p.H;
  RowSum<WARP, MAXT> row_sum{red, nw, 0};
  auto col = [&](int j) { return (j * nthr + tid) * 8; };
  using W = Raw<uint16_t>;
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
  Raw<RT> rn[NV] = {};
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
    float r[NV][8];
    float v[NV][8];
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
      for (int e = 0; e < 8; ++e) {
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
          for (int e = 0; e < 8; ++e) s = fmaf(v[j][e], v[j][e], s);
        inv = rsqrtf(row_sum(s) * inv_h + p.eps);
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (col(j) >= p.H) continue;
        const W w = kAhead ? wpost[j] : load_w(p.post_weight, j);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
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
        if (col(j) < p.H) store_vals<8>(op + col(j), r[j]);
    }
    if (!p.out && !p.out_q) continue;
    if (p.pre_weight) {
      s = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(r[j][e], r[j][e], s);
      const float inv = rsqrtf(row_sum(s) * inv_h + p.eps);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (col(j) >= p.H) continue;
        const W w = kAhead ? wpre[j] : load_w(p.pre_weight, j);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[j][e] = r[j][e] * inv * (p.weight_offset + w.at(e));
      }
    }
    if (p.out) {
      uint16_t* op = p.out + row * p.out_ld;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (col(j) < p.H) store_vals<8>(op + col(j), r[j]);
    }
    if (p.out_q) {
      uint8_t* qp = p.out_q + row * p.out_q_ld;
      float* sp = p.out_scale + row * ((p.H + kQuantGroup - 1) / kQuantGroup);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float a = 0.0f;  // values past H are 0
#pragma unroll
        for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(r[j][e]));
        // a group is 16 neighbouring lanes
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        const int c = col(j);
        if (c >= p.H) continue;
        const QuantScale qs = quant_scale(a);
        *reinterpret_cast<uint2*>(qp + c) =
            make_uint2(quant4(r[j][0], r[j][1], r[j][2], r[j][3], qs),
                       quant4(r[j][4], r[j][5], r[j][6], r[j][7], qs));
        if (c % kQuantGroup == 0) sp[c / kQuantGroup] = qs.s;
      }
    }
  }
}

// -------------------------------------------------- rows of any alignment
// A row of H values on its way to shared memory.  Its 16-byte pieces are
// copied asynchronously to where they lie within 16 bytes, so that value i is
// value `lead + i` of the buffer; the few values before the first piece and
// after the last go through a register of the first 16 threads.
template <typename T>
struct RowCopy {
  static constexpr int kPiece = 16 / (int)sizeof(T);
  int lead, head, pieces;
  __device__ __forceinline__ RowCopy(const T* p, int H) {
    lead = (int)(reinterpret_cast<uintptr_t>(p) & 15) / (int)sizeof(T);
    head = lead ? min(H, kPiece - lead) : 0;
    pieces = (H - head) / kPiece;
  }
  // the value outside the pieces that a thread carries, or -1
  __device__ __forceinline__ int edge(int H) const {
    const int t = threadIdx.x;
    const int i = t < 8 ? t : head + pieces * kPiece + t - 8;
    return t < 8 ? (t < head ? i : -1) : (t < 16 && i < H ? i : -1);
  }
  __device__ __forceinline__ T start(T* buf, const T* p, int H) const {
    const uint32_t dst = smem_u32(buf + lead + head);
    for (int c = threadIdx.x; c < pieces; c += blockDim.x) cp_async16(dst + c * 16, p + head + c * kPiece);
    const int e = edge(H);
    return e >= 0 ? p[e] : T(0);
  }
  __device__ __forceinline__ void finish(T* buf, T edge_value, int H) const {
    const int e = edge(H);
    if (e >= 0) buf[lead + e] = edge_value;
  }
};
__host__ __device__ constexpr int any_row_bytes(int H, int size) { return (H * size + 16 + 15) / 16 * 16; }

// Rows of odd widths, strides or addresses: a CTA walks rows, each staged in
// shared memory by 16-byte copies (in two buffers, the next row's copies beside
// this row's work, where two fit) and written value by value.  Value j of a
// thread is value 32 NV warp + 32 j + lane, so a warp holds whole groups of 128.
// 601 x 1999 fp32 takes 6.3 us, 4096 x 2047 bf16 with codes 29 us (2.6 TB/s),
// 1000 x 5001 16 us; with loads of single values in place of the copies, too few
// bytes were in flight: 8.5, 51 and 62 us.  16 values a thread took 8.3, 30 and
// 16 us, 4 values 8.0, 42 and 21.
template <int NV, int MAXT, bool GATED, typename RT>
__global__ void __launch_bounds__(MAXT, kAnyResident / MAXT) block_norm_any_kernel(const oes_block_norm p, int bufs) {
  pdl_begin();
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float red[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int H = p.H;
  const float inv_h = 1.0f / (float)H;
  RowSum<false, MAXT> row_sum{red, (int)(blockDim.x >> 5), 0};
  const bool elem = GATED && p.gate_kind == OES_GATE_ELEMENT;
  const int r_bytes = any_row_bytes(H, sizeof(RT)), y_bytes = p.y ? any_row_bytes(H, 2) : 0;
  const int buf_bytes = r_bytes + y_bytes + (elem ? any_row_bytes(H, 2) : 0);
  const RT* rg = static_cast<const RT*>(p.residual);
  const uint16_t* gg = static_cast<const uint16_t*>(p.gate);
  RT r_edge = RT(0);
  uint16_t y_edge = 0, g_edge = 0;
  float gn = 0.0f;
  auto start = [&](int64_t row, int b) {
    if (row >= p.T) return;
    uint8_t* buf = smem + b * buf_bytes;
    const RT* rp = rg + row * p.residual_ld;
    r_edge = RowCopy<RT>(rp, H).start(reinterpret_cast<RT*>(buf), rp, H);
    if (p.y) {
      const uint16_t* yp = p.y + row * p.y_ld;
      y_edge = RowCopy<uint16_t>(yp, H).start(reinterpret_cast<uint16_t*>(buf + r_bytes), yp, H);
    }
    if (elem) {
      const uint16_t* gp = gg + row * p.gate_ld;
      g_edge = RowCopy<uint16_t>(gp, H).start(reinterpret_cast<uint16_t*>(buf + r_bytes + y_bytes), gp, H);
    }
    if (p.gate_kind == OES_GATE_TOKEN) gn = static_cast<const float*>(p.gate)[row * p.gate_ld];
  };
  const int c0 = warp * 32 * NV + lane;
  auto col = [&](int j) { return c0 + 32 * j; };
  int b = 0;
  start(blockIdx.x, 0);
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    uint8_t* buf = smem + b * buf_bytes;
    RT* rb = reinterpret_cast<RT*>(buf);
    uint16_t* yb = reinterpret_cast<uint16_t*>(buf + r_bytes);
    uint16_t* gb = reinterpret_cast<uint16_t*>(buf + r_bytes + y_bytes);
    cp_async_wait_all();
    const RowCopy<RT> rc(rg + row * p.residual_ld, H);
    const RowCopy<uint16_t> yc(p.y + row * p.y_ld, H), gc(gg + row * p.gate_ld, H);
    rc.finish(rb, r_edge, H);
    if (p.y) yc.finish(yb, y_edge, H);
    if (elem) gc.finish(gb, g_edge, H);
    const float gt = gn;
    __syncthreads();  // the row is here, and every thread is done with the one before
    if (bufs == 2) {
      b ^= 1;
      start(row + gridDim.x, b);
    }
    float r[NV], v[NV];
    uint16_t w[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool in = col(j) < H;
      r[j] = in ? widen(rb[rc.lead + col(j)]) : 0.0f;
      v[j] = in && p.y ? widen(yb[yc.lead + col(j)]) : 0.0f;
    }
    auto load_w = [&](const uint16_t* wp) {
#pragma unroll
      for (int j = 0; j < NV; ++j) w[j] = wp && col(j) < H ? wp[col(j)] : (uint16_t)0;
    };
    float s = 0.0f;
    if (p.y) {
      float k = p.residual_scale;
      if (p.gate_kind == OES_GATE_TOKEN) k *= p.gate_sigmoid ? sigmoid_f32(gt) : gt;
      if (p.post_weight) {
        load_w(p.post_weight);
#pragma unroll
        for (int j = 0; j < NV; ++j) s = fmaf(v[j], v[j], s);
        const float inv = rsqrtf(row_sum(s) * inv_h + p.eps);
#pragma unroll
        for (int j = 0; j < NV; ++j) v[j] = v[j] * inv * (p.weight_offset + widen(w[j]));
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (col(j) >= H) continue;
        if (GATED) {
          const float g = widen(elem ? gb[gc.lead + col(j)] : gg[col(j)]);
          v[j] *= p.gate_sigmoid ? sigmoid_f32(g) : g;
        }
        r[j] = fmaf(k, v[j], r[j]);
      }
    }
    if (p.out_residual) {
      RT* op = static_cast<RT*>(p.out_residual) + row * p.out_residual_ld;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (col(j) < H) narrow(op + col(j), r[j]);
    }
    if (p.out || p.out_q) {
      if (p.pre_weight) {
        load_w(p.pre_weight);
        s = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) s = fmaf(r[j], r[j], s);
        const float inv = rsqrtf(row_sum(s) * inv_h + p.eps);
#pragma unroll
        for (int j = 0; j < NV; ++j) r[j] = r[j] * inv * (p.weight_offset + widen(w[j]));
      }
      if (p.out) {
        uint16_t* op = p.out + row * p.out_ld;
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (col(j) < H) narrow(op + col(j), r[j]);
      }
      if (p.out_q) {
        uint8_t* qp = p.out_q + row * p.out_q_ld;
        float* sp = p.out_scale + row * ((H + kQuantGroup - 1) / kQuantGroup);
#pragma unroll
        for (int n = 0; n < NV / 4; ++n) {  // values past H are 0
          float a = 0.0f;
#pragma unroll
          for (int j = 4 * n; j < 4 * n + 4; ++j) a = fmaxf(a, col(j) < H ? fabsf(r[j]) : 0.0f);
#pragma unroll
          for (int o = 16; o >= 1; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
          const QuantScale qs = quant_scale(a);
#pragma unroll
          for (int j = 4 * n; j < 4 * n + 4; ++j)
            if (col(j) < H) qp[col(j)] = quant1(r[j], qs);
          if (lane == 0 && col(4 * n) < H) sp[col(4 * n) / kQuantGroup] = qs.s;
        }
      }
    }
    if (bufs == 1) {
      __syncthreads();  // every thread is done with the row
      start(row + gridDim.x, 0);
    }
  }
}

template <int NV, bool WARP, int MAXT>
int launch_norm(const oes_block_norm& p, int threads, cudaStream_t stream) {
  const int rows = WARP ? threads / 32 : 1;
  const int64_t want = ceil_div64(p.T, rows);
  // about the CTAs that are resident at once, so that each walks its rows
  const int grid = (int)std::min<int64_t>(want, (int64_t)num_sms() * std::max(1, kNormResident / threads));
  auto go = [&](auto kernel) { launch_kernel(kernel, grid, threads, 0, stream, p); };
  const bool gated = p.gate_kind >= OES_GATE_CHANNEL;
  if (p.dtype == OES_BF16) {
    if (gated) go(block_norm_kernel<NV, WARP, MAXT, true, uint16_t>);
    else go(block_norm_kernel<NV, WARP, MAXT, false, uint16_t>);
  } else {
    if (gated) go(block_norm_kernel<NV, WARP, MAXT, true, float>);
    else go(block_norm_kernel<NV, WARP, MAXT, false, float>);
  }
  OES_CHECK_LAUNCH("block_norm_kernel");
  return OES_OK;
}

template <int NV, int MAXT>
int launch_any(const oes_block_norm& p, cudaStream_t stream) {
  const int threads = ceil_div(p.H, 32 * NV) * 32;
  const int row = any_row_bytes(p.H, p.dtype == OES_BF16 ? 2 : 4) + (p.y ? any_row_bytes(p.H, 2) : 0) +
                  (p.gate_kind == OES_GATE_ELEMENT ? any_row_bytes(p.H, 2) : 0);
  const int bufs = 2 * row <= kAnySmem ? 2 : 1;
  const int per_sm = std::max(1, std::min(std::min(kAnyResident / threads, 32), kAnySmem / (bufs * row + 1024)));
  // a CTA a row up to four rows for each resident CTA: few rows a CTA would leave
  // some with one more than others (4096 x 499: 13.3 us, 16.0 in walked rows;
  // 4096 x 2047 at eight rows: 31.9, 29.0 walked)
  const int64_t resident = (int64_t)num_sms() * per_sm;
  const int grid = (int)(p.T <= 4 * resident ? p.T : resident);
  auto go = [&](auto kernel) {
    const int rc = set_max_dynamic_smem((const void*)kernel, bufs * row, "block_norm_any_kernel");
    if (rc) return rc;
    launch_kernel(kernel, grid, threads, bufs * row, stream, p, bufs);
    OES_CHECK_LAUNCH("block_norm_any_kernel");
    return (int)OES_OK;
  };
  const bool gated = p.gate_kind >= OES_GATE_CHANNEL;
  if (p.dtype == OES_BF16)
    return gated ? go(block_norm_any_kernel<NV, MAXT, true, uint16_t>) : go(block_norm_any_kernel<NV, MAXT, false, uint16_t>);
  return gated ? go(block_norm_any_kernel<NV, MAXT, true, float>) : go(block_norm_any_kernel<NV, MAXT, false, float>);
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
  if (vec) {
    auto up = [](int n, int m) { return (n + m - 1) / m * m; };
    const int c = p.H / 8, half = up(ceil_div(c, 2), 32);  // 16 values a thread
    if (c <= 64) return launch_norm<2, true, 128>(p, 128, stream);
    if (half <= 128) return launch_norm<2, false, 128>(p, half, stream);
    if (half <= 256) return launch_norm<2, false, 256>(p, half, stream);
    if (half <= 512) return launch_norm<2, false, 512>(p, half, stream);
    return launch_norm<2, false, 1024>(p, half, stream);
  }
  if (p.H <= 2048) return launch_any<8, 256>(p, stream);
  if (p.H <= 4096) return launch_any<8, 512>(p, stream);
  return launch_any<16, 1024>(p, stream);
}
