// moe_layer_few_tokens: a whole mixture-of-experts layer for up to 16 tokens in
// two launches.
//
//   out[t] = sum_j w[t, j] W2_e (silu(Wg_e x_t) * (Wu_e x_t)),   e = ids[t, j]
//
// A few tokens reach a few experts each, so the layer is a stream of those
// experts' weights (one token x 10 of 512 FP8 experts: 47 MB, 7 us at the copy
// rate), and everything around that stream is latency.
//
//   few_up_kernel    routes the tokens and makes the chunk's tables in every CTA
//                    (waiting for a kernel that does costs more), then h: a unit is
//                    8 rows of I of one block, whose 8 gate rows and same 8 up rows
//                    are the 16 rows of one matrix instruction, so that a lane has
//                    both factors of its h.
//   few_down_kernel  a CTA owns up to 16 rows of the output at a time and goes
//                    through all blocks for them, its warps sharing the (block, step
//                    of K); the weighted sum over a token's routes is the
//                    accumulator.  It takes the tables from the first kernel, and
//                    its CTAs fill their queues with W2 while the last of that
//                    kernel's still run.
//
// A block is one expert with at most one route of each token.  In the first kernel
// column c of the matrix instruction is token c, in the second the columns are the parts
// of the block's rows of h.  An expert that a token lists twice gets a second block for
// the second route.
//
// Weights go from memory into a queue of each lane's own (16-byte asynchronous
// copies, read back by the same lane), so a warp keeps its next steps in
// flight without registers and without a barrier.  The instructions are the
// warp-wide m16n8k16, whose tensor work at 8 columns is a small part of what the
// stream takes (9 to 19 % of the pipe); the grouped GEMM's tcgen05 tiles (128 weight rows,
// operands through shared memory and TMEM) reach 9 to 30 % of the copy rate for 1 to 64
// tokens of NVFP4 experts, held up by their set-up and hand-offs.
//
// Measured (10 of 512 experts of 2048 x 768, replayed from a graph): 1 token FP8 16.8 us
// (2.8 TB/s), bf16 21.9 us (4.3); 4 tokens NVFP4 38.9 us (2.6); 16 tokens bf16 207 to 219 us (6.0 to
// 6.3 TB/s, 88 to 93 % of the copy rate, by GPU), FP8 138 us (4.8), NVFP4 143 us (2.6).  16 bf16 tokens
// are bound by memory; the 8- and 4-bit formats by the instructions that decode and multiply (issue
// slots 37 to 52 % busy); one token by latency: 4.4 us to the first weights (logits, top-k, tables,
// slots), 2 to 3 from one kernel to the next, 1.3 for the last sums.
//
// Weights are exact in 16 bits: bf16 as they are; e4m3 as f16, their block scales on
// the fp32 sums of each 128 of K; e2m1 x e4m3 as f16, the global scale on the sums.
// h is fp32.  For bf16 weights x is taken as it is, and h as three bf16 numbers, which hold
// all of it; for the others x is f16 numbers with a power of two for each 128, exact
// unless 2^31 smaller than the largest of them, and h two such (f16_group), of 22 bits.
// (h of 16 and of 11 bits, as it was: of the 16-token case's results 383 of 131072 were not
// the 64-bit sums' roundings, now 35, of one token's in FP8 856 of 8192, now 1; fp32 matrix
// products of torch miss 113 and 5.)  An instruction's sum is what the tensor core keeps of
// it, so no chain of them goes past a step: steps are added up in fp32, as are a token's
// routes, and out is rounded once.
#include <algorithm>

#include "common.cuh"
#include "fp8_dev.cuh"
#include "gemm_types.h"
#include "internal.h"
#include "route_dev.cuh"
#include "warp_mma.cuh"

namespace oes {

namespace {

__host__ __device__ constexpr int cdiv(int a, int b) { return (a + b - 1) / b; }

constexpr int kMaxTokens = 16;    // of a call
constexpr int kFusedExperts = 512;  // most experts that the kernels route themselves
constexpr int kRowTile = 16;
constexpr int W = 16;  // warps of a CTA

// Weight formats.  A step is what a warp takes from its queue at a time: kStepK
// values of 16 rows, kChunks x 16 bytes a lane, the step's scales behind them; of
// the activations a lane needs 2 x kB x 16 bytes for each column, half a step at a
// time.  kF16: the activations are f16 numbers with a power of two for each 128
// (see f16_group), else bf16.
template <int WF>
struct Fmt;
template <>
struct Fmt<OES_WFMT_BF16> {
  static constexpr int kStepK = 64, kRowBytes = 128, kChunks = 4, kB = 1, kXPad = 64;
  static constexpr int kScale = 0;
  static constexpr bool kF16 = false;
};
template <>
struct Fmt<OES_WFMT_FP8> {
  static constexpr int kStepK = 128, kRowBytes = 128, kChunks = 4, kB = 2, kXPad = 16;
  static constexpr int kScale = 64;  // 16 fp32, one a row (few_up: gate, up)
  static constexpr bool kF16 = true;
};
template <>
struct Fmt<OES_WFMT_NVFP4> {
  static constexpr int kStepK = 128, kRowBytes = 64, kChunks = 2, kB = 2, kXPad = 16;
  static constexpr int kScale = 128;  // [2 x 64 of K][16 rows][4] e4m3
  static constexpr bool kF16 = true;
};
template <int WF>
__host__ __device__ constexpr int entry_bytes() {
  return Fmt<WF>::kChunks * 512 + Fmt<WF>::kScale;
}

// Bytes of a value of h.
__host__ __device__ constexpr int h_value_bytes(int wfmt) { return wfmt == OES_WFMT_BF16 ? 6 : 4; }

struct FewParams {
  const uint8_t* pool;
  int64_t row_bytes;
  const int32_t* e2s;
  int E, S, H, I, T, k;
  const uint16_t* x;
  const void* logits;  // NULL: ids and weights are given
  int logits_bf16;
  int32_t* ids;
  float* weights;
  void* h;  // [T k, I] (store_h)
  uint16_t* out;
  int32_t* status;
  int64_t s13, w2, s2, gs;  // sections of an expert row
  uint8_t* tables;          // from few_up to few_down: the number of blocks, whether the tables are there,
                            // and from byte 16 on the tables
  int x_ld;                 // bytes of a row of x in shared memory
  int rows_cta;             // few_down: rows of out a CTA owns
};

// The chunk's tables, in shared memory.  A block's first route leads it.  few_down takes
// the first down_tables_bytes() of them.
struct Tables {
  float* w;        // [R]
  int32_t* slot;   // [blocks]
  uint32_t* has;   // [blocks] which tokens have a route in the block
  int16_t* order;  // [R] the routes that count, block after block, each by its tokens
  int16_t* cum;    // [blocks] a block's first place there
  int32_t* ids;    // [R], few_up alone from here on
  int32_t* lead;   // [R] first route of the route's block, -1 for one that does not count
  int32_t* blk;    // [R] block of a leading route
  int16_t* route;  // [blocks][8 NG] route of each token in the block, or -1
  __device__ __forceinline__ Tables(uint8_t* base, int R) {
    w = reinterpret_cast<float*>(base);
    slot = reinterpret_cast<int32_t*>(w + R);
    has = reinterpret_cast<uint32_t*>(slot + R);
    order = reinterpret_cast<int16_t*>(has + R);
    cum = order + R;
    ids = reinterpret_cast<int32_t*>(base + R * 16);
    lead = ids + R;
    blk = lead + R;
    route = reinterpret_cast<int16_t*>(blk + R);
  }
};
__host__ __device__ constexpr int down_tables_bytes(int R) { return R * 16; }
__host__ __device__ constexpr int tables_bytes(int R, int ng) { return R * (28 + 16 * ng); }

// One token's top-k by one warp, the ids and weights of topk_row_filtered bit for bit
// (the same threshold, the same order of the candidates, topk_write), made for a single
// row's latency: candidates find their places by ballots instead of a counter in
// shared memory, whose round trips a lone warp has nothing to hide behind, and rank
// themselves against broadcasts.  E <= 512; cand: 32 entries of the warp's own.
template <typename LT>
__device__ __forceinline__ void topk_few(const LT* __restrict__ row, int E, int k, int lane, int32_t* ids, float* w,
                                         uint64_t* cand) {
  constexpr int Q = kFusedExperts / 32;
  float v[Q];
#pragma unroll
  for (int j = 0; j < Q; ++j) {
    v[j] = __int_as_float(0x7fffffff);  // NaN: no expert
    if (lane + 32 * j < E) v[j] = load_logit(row + lane + 32 * j);
  }
  float m = -INFINITY;  // fmaxf skips NaN
#pragma unroll
  for (int j = 0; j < Q; ++j) m = fmaxf(m, v[j]);
  // the lane maxima in descending order; tau the k-th
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int d = size >> 1; d > 0; d >>= 1) {
      const float o = __shfl_xor_sync(0xffffffffu, m, d);
      m = (((lane & d) == 0) == ((lane & size) == 0)) ? fmaxf(m, o) : fminf(m, o);
    }
  const float tau = __shfl_sync(0xffffffffu, m, k - 1);
  int n = 0;
  if (tau > -INFINITY) {
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      const uint32_t at = __ballot_sync(0xffffffffu, v[j] >= tau);
      const int place = n + __popc(at & ((1u << lane) - 1));
      if (v[j] >= tau && place < 32)  // larger key first, then the lower id
        cand[place] = ((uint64_t)logit_key(v[j]) << 32) | (uint32_t)~(lane + 32 * j);
      n += __popc(at);
    }
  }
  if (n == 0 || n > 32) {  // few numbers above -inf, or many equal ones: in rounds
    uint32_t key[Q];
#pragma unroll
    for (int j = 0; j < Q; ++j) key[j] = lane + 32 * j < E ? logit_key(v[j]) : 0u;
    topk_rounds<Q, 1>(key, k, lane, ids, w);
    return;
  }
  __syncwarp();
  const uint64_t mine = lane < n ? cand[lane] : 0;
  int r = 0;
#pragma unroll 8
  for (int c = 0; c < n; ++c) r += cand[c] > mine;
  __syncwarp();
  if (lane < n && r < k) cand[r] = mine;
  __syncwarp();
  const uint64_t won = lane < k ? cand[lane] : 0;
  topk_write((uint32_t)(won >> 32), ~(uint32_t)won, k, lane, ids, w);
}

// Routing and tables, by the whole CTA; returns the number of blocks.  One CTA
// writes the router's outputs and the status (`first`).  scratch: shared memory, one
// word an expert, two with logits.  Beside the routing, the warps that have no token
// run side(i, n), i of n threads (with a token for every warp, all do, behind it).
template <int NG, typename Side>
__device__ __forceinline__ int few_tables(const FewParams& p, const Tables& tb, uint8_t* scratch, bool first,
                                          const Side& side) {
  __shared__ uint64_t cand[kMaxTokens][32];
  __shared__ int s_leads[OES_FEW_TOKENS_MAX * OES_MAX_TOPK / 32 + 1];
  __shared__ int s_one;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x, nw = nt >> 5;
  const int R = p.T * p.k, chunks = cdiv(R, 32);
  int32_t* fst = reinterpret_cast<int32_t*>(scratch);  // [E] the first route to each expert
  int32_t* map = fst + p.E;                            // [E] the slot map, with logits
  const int routers = p.logits && p.T < nw ? p.T : 0;
  auto init = [&](int i0, int n) {
    for (int i = i0; i < p.E; i += n) {
      fst[i] = 0x7FFFFFFF;
      if (p.logits) cp_async4_take(smem_u32(map + i), p.e2s + i, true);
    }
    for (int i = i0; i < R * 4 * NG; i += n) reinterpret_cast<int32_t*>(tb.route)[i] = -1;
    for (int i = i0; i < R; i += n) {
      tb.has[i] = 0u;
      if (!p.logits) {
        tb.ids[i] = __ldcg(p.ids + i);
        tb.w[i] = __ldcg(p.weights + i);
      }
    }
    side(i0, n);
  };
  if (warp >= routers && routers > 0) {
    init(tid - routers * 32, nt - routers * 32);
  } else if (p.logits) {
    for (int t = warp; t < p.T; t += nw) {
      int32_t* ids = tb.ids + t * p.k;
      float* w = tb.w + t * p.k;
      if (p.logits_bf16)
        topk_few(static_cast<const uint16_t*>(p.logits) + (size_t)t * p.E, p.E, p.k, lane, ids, w, cand[warp]);
      else
        topk_few(static_cast<const float*>(p.logits) + (size_t)t * p.E, p.E, p.k, lane, ids, w, cand[warp]);
    }
  }
  if (routers == 0) init(tid, nt);
  cp_async_wait<0>();
  __syncthreads();
  if (p.logits && p.T == 1) {
    // one token, distinct experts: where all have slots, block r is route r
    if (warp == 0) {
      const int e = lane < R ? tb.ids[lane] : 0;
      const int slot = lane < R ? map[e] : 0;
      const bool all = __all_sync(0xffffffffu, slot >= 0 && slot < p.S);
      if (all && lane < R) {
        tb.slot[lane] = slot;
        tb.lead[lane] = tb.blk[lane] = lane;
        tb.has[lane] = 1u;
        tb.route[lane * 8 * NG] = (int16_t)lane;
        if (first) {
          p.ids[lane] = e;
          p.weights[lane] = tb.w[lane];
        }
      }
      if (lane == 0) s_one = all;
    }
    __syncthreads();
    if (s_one) return R;
  }
  for (int r = tid; r < R; r += nt) {
    const int e = tb.ids[r];
    if (first && p.logits) {
      p.ids[r] = e;
      p.weights[r] = tb.w[r];
    }
    int n = -1;  // this is the token's route number n to e
    if (e >= 0 && e < p.E) {
      const int slot = p.logits ? map[e] : __ldcg(p.e2s + e);
      if (slot >= 0 && slot < p.S) {
        n = 0;
        if (!p.logits)
          for (int i = r / p.k * p.k; i < r; ++i) n += tb.ids[i] == e;
        if (n == 0) atomicMin(&fst[e], r);
        tb.blk[r] = slot;  // a leading route's, until the blocks are numbered
      } else if (first) {
        set_status(p.status, OES_DEV_BAD_ID);
      }
    }
    tb.lead[r] = n;
  }
  __syncthreads();
  // the block's first route is the first token's that has as many to e
  for (int c = warp; c < chunks; c += nw) {
    const int r = c * 32 + lane;
    int lead = -1;
    if (r < R) {
      const int n = tb.lead[r];
      if (n >= 0) {
        const int e = tb.ids[r];
        lead = r;
        if (n == 0) {
          lead = fst[e];
        } else {
          for (int u = 0; u < r / p.k && lead == r; ++u) {
            int m = 0;
            for (int i = u * p.k; i < (u + 1) * p.k; ++i)
              if (tb.ids[i] == e && m++ == n) {
                lead = i;
                break;
              }
          }
        }
      }
      tb.lead[r] = lead;
    }
    const uint32_t m = __ballot_sync(0xffffffffu, r < R && lead == r);
    if (lane == 0) s_leads[c] = __popc(m);
  }
  __syncthreads();
  for (int c = warp; c < chunks; c += nw) {
    const int r = c * 32 + lane;
    const bool is = r < R && tb.lead[r] == r;
    const uint32_t m = __ballot_sync(0xffffffffu, is);
    const int before = __reduce_add_sync(0xffffffffu, lane < c ? s_leads[lane] : 0);
    if (is) {
      const int b = before + __popc(m & ((1u << lane) - 1));
      tb.slot[b] = tb.blk[r];
      tb.blk[r] = b;
    }
  }
  __syncthreads();
  for (int r = tid; r < R; r += nt) {
    const int lead = tb.lead[r];
    if (lead >= 0) {
      const int b = tb.blk[lead], t = r / p.k;
      tb.route[b * 8 * NG + t] = (int16_t)r;
      atomicOr(&tb.has[b], 1u << t);
    }
  }
  __syncthreads();
  int nb = 0;
  for (int c = 0; c < chunks; ++c) nb += s_leads[c];
  return nb;
}

// The routes that count in the order of their blocks, for few_down.
template <int NG>
__device__ void few_order(const FewParams& p, const Tables& tb, int nb) {
  __shared__ int s_sums[OES_FEW_TOKENS_MAX * OES_MAX_TOPK / 32 + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
  const int chunks = cdiv(nb, 32), nw = nt >> 5;
  for (int c = warp; c < chunks; c += nw) {
    const int b = c * 32 + lane;
    const int n = b < nb ? __popc(tb.has[b]) : 0;
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += u;
    }
    if (b < nb) tb.cum[b] = (int16_t)(sum - n);
    if (lane == 31) s_sums[c] = sum;
  }
  __syncthreads();
  for (int c = warp; c < chunks; c += nw) {
    const int before = __reduce_add_sync(0xffffffffu, lane < c ? s_sums[lane] : 0);
    if (c * 32 + lane < nb) tb.cum[c * 32 + lane] += (int16_t)before;
  }
  __syncthreads();
  for (int i = tid; i < nb * 8 * NG; i += nt) {
    const int b = i / (8 * NG), t = i % (8 * NG), r = tb.route[i];
    if (r >= 0) tb.order[tb.cum[b] + __popc(tb.has[b] & ((1u << t) - 1))] = (int16_t)r;
  }
  __syncthreads();
}

// The matrix instructions of half a step: the lane's weights from its queue entry,
// added onto d (row g and g + 8, columns 2t and 2t + 1, of each 8 columns), or FRESH from
// zero.  B are the lane's values of the columns.
template <int WF, int NG, bool FRESH>
__device__ __forceinline__ void half_mma(uint32_t entry, int hh, const uint4 (&B)[NG][Fmt<WF>::kB], float (&d)[NG][4]) {
  const int lane = threadIdx.x & 31;
  const uint32_t mine = entry + lane * 16;
  if constexpr (WF == OES_WFMT_BF16) {
    const uint4 a = lds128(mine + hh * 1024), b = lds128(mine + hh * 1024 + 512);
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      mma_16816<false, FRESH>(d[n], a.x, b.x, a.y, b.y, B[n][0].x, B[n][0].y);
      mma_16816<false>(d[n], a.z, b.z, a.w, b.w, B[n][0].z, B[n][0].w);
    }
  } else if constexpr (WF == OES_WFMT_FP8) {
    const uint4 a = lds128(mine + hh * 1024), b = lds128(mine + hh * 1024 + 512);
    const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t a0, a2, a1, a3;
      e4m3x4_f16x4(aw[i], a0, a2);
      e4m3x4_f16x4(bw[i], a1, a3);
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        const uint4& v = B[n][i >> 1];
        if (i == 0) mma_16816<true, FRESH>(d[n], a0, a1, a2, a3, v.x, v.y);
        else mma_16816<true>(d[n], a0, a1, a2, a3, i & 1 ? v.z : v.x, i & 1 ? v.w : v.y);
      }
    }
  } else {
    const int g = lane >> 2, t = lane & 3;
    const uint2 a = lds64(mine + hh * 8), b = lds64(mine + 512 + hh * 8);
    const uint32_t aw[2] = {a.x, a.y}, bw[2] = {b.x, b.y};
    // the lane's 32 values have the scales of groups 2t and 2t + 1 of the step
    const uint32_t sc = entry + 1024 + (t >> 1) * 64 + g * 4;
    const uint32_t sa = e4m3x2_f16x2((lds32(sc) >> (16 * (t & 1))) & 0xFFFFu);
    const uint32_t sb = e4m3x2_f16x2((lds32(sc + 32) >> (16 * (t & 1))) & 0xFFFFu);
    const uint32_t fa = __byte_perm(sa, 0, hh ? 0x3232 : 0x1010), fb = __byte_perm(sb, 0, hh ? 0x3232 : 0x1010);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t oa[4], ob[4];
      e2m1x8_f16x8(aw[i], oa);
      e2m1x8_f16x8(bw[i], ob);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        oa[j] = mul_f16x2(oa[j], fa);
        ob[j] = mul_f16x2(ob[j], fb);
      }
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        if (i == 0) mma_16816<true, FRESH>(d[n], oa[0], ob[0], oa[1], ob[1], B[n][i].x, B[n][i].y);
        else mma_16816<true>(d[n], oa[0], ob[0], oa[1], ob[1], B[n][i].x, B[n][i].y);
        mma_16816<true>(d[n], oa[2], ob[2], oa[3], ob[3], B[n][i].z, B[n][i].w);
      }
    }
  }
}

// First value along K, within a step, of 16-byte piece i of the lane's half hh.
template <int WF>
__device__ __forceinline__ int piece_k(int hh, int i) {
  const int t = threadIdx.x & 3;
  return WF == OES_WFMT_BF16 ? 32 * hh + 8 * t : WF == OES_WFMT_FP8 ? 64 * hh + 16 * t + 8 * i : 32 * t + 16 * hh + 8 * i;
}

// The lane's copies of one step: 16 rows' kRowBytes, at r0 (row g) and r1 (row g + 8) for
// this lane; n0, n1: 16, or 0 for a row that is absent and becomes zeros.
template <int WF>
__device__ __forceinline__ void step_copy(uint32_t entry, const uint8_t* r0, const uint8_t* r1, int n0, int n1) {
  const uint32_t mine = entry + (threadIdx.x & 31) * 16;
#pragma unroll
  for (int hh = 0; hh < Fmt<WF>::kChunks / 2; ++hh) {
    cp_async16_part(mine + hh * 1024, r0 + hh * 64, n0);
    cp_async16_part(mine + hh * 1024 + 512, r1 + hh * 64, n1);
  }
}
// The same for a row's last step of `left` bytes: what is past them becomes zeros, and
// nothing is read for it (any readable address stands in).
template <int WF>
__device__ __forceinline__ void step_copy_last(uint32_t entry, const uint8_t* r0, const uint8_t* r1, int n0, int n1,
                                               int left, const uint8_t* any) {
  const int lane = threadIdx.x & 31;
  const uint32_t mine = entry + lane * 16;
#pragma unroll
  for (int hh = 0; hh < Fmt<WF>::kChunks / 2; ++hh) {
    const bool in = hh * 64 + 16 * (lane & 3) < left;
    cp_async16_part(mine + hh * 1024, in ? r0 + hh * 64 : any, in ? n0 : 0);
    cp_async16_part(mine + hh * 1024 + 512, in ? r1 + hh * 64 : any, in ? n1 : 0);
  }
}

// Activations for 8- and 4-bit weights: f16 numbers with one power of two for each
// 128 along K, chosen so that the largest is in [2^14, 2^15).  The sums of a step
// span just such 128, so the factor goes to the sums.  A number keeps 11
// significant bits down to 2^-29 of its group's largest (a bf16 number all of its 8 down to
// 2^-31), and nothing leaves f16's range, whatever the activations' own.  TWO: a second
// number holds what the first one's 11 bits left, together 22 bits, down to 2^-17 of the
// largest (2^-39 of the largest is the least difference).  The group is 16 neighbouring
// lanes' 8 values each; returns the factor that undoes it.  A NaN stays one and counts for
// nothing else, an infinity stays one.
template <bool TWO>
__device__ __forceinline__ float f16_group(const float (&v)[8], uint4& first, uint4& second) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const uint32_t ex = min(max(__float_as_uint(m) >> 23, 27u), 254u);  // 2^-100 at least
  const float f = __uint_as_float((268u - ex) << 23);
  uint32_t a[4], b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo = v[2 * i] * f, hi = v[2 * i + 1] * f;
    if (TWO) {
      const float l = __uint_as_float(__float_as_uint(lo) & 0xFFFFE000u), h = __uint_as_float(__float_as_uint(hi) & 0xFFFFE000u);
      asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(b[i]) : "f"(hi - h), "f"(lo - l));
      if (m == INFINITY) b[i] = 0u;  // what an infinity leaves is none of its difference's NaN
      lo = l;
      hi = h;
    }
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(a[i]) : "f"(hi), "f"(lo));
  }
  first = make_uint4(a[0], a[1], a[2], a[3]);
  if (TWO) second = make_uint4(b[0], b[1], b[2], b[3]);
  return __uint_as_float((ex - 14u) << 23);
}

// One value of a route's h, for the down kernel: fp32, or for bf16 weights as three bf16 numbers, each what
// rounding to those before left (24 significant bits, all that fp32 has), the first ones of 64 values
// before their second and third ones.
template <int WF>
__device__ __forceinline__ void store_h(const FewParams& p, int r, int i, float v) {
  if constexpr (Fmt<WF>::kF16) {
    static_cast<float*>(p.h)[(int64_t)r * p.I + i] = v;
  } else {
    constexpr int K = Fmt<WF>::kStepK;
    const uint32_t one = f32_bf16(v);
    // an infinity leaves nothing (and not the NaN of its difference)
    const float left = fabsf(bf16_f32(one)) < INFINITY ? v - bf16_f32(one) : 0.0f;
    const uint32_t two = f32_bf16(left);
    uint16_t* to = static_cast<uint16_t*>(p.h) + ((int64_t)r * p.I + i / K * K) * 3 + i % K;
    to[0] = (uint16_t)one;
    to[K] = (uint16_t)two;
    to[2 * K] = (uint16_t)f32_bf16(left - bf16_f32(two));
  }
}

template <int V>
struct Int {
  static constexpr int value = V;
};

// ------------------------------------------------------------------ gate, up
// A unit is 8 rows of I of a block.  The chunk's units are dealt out to the CTAs in
// runs, and a CTA's to its teams of KS warps, which share the unit's K range.  KS 1: a
// lane ends with both factors of its h, and no barrier follows the tables.  (With eight
// warps a unit throughout, 16 tokens x 10 of 512 FP8 experts took 243 us, with one 166.)
// More where there are few units (see launch_few): one warp keeps 8 KB in flight.
template <int WF, int NG, int KS, int S>
__global__ void __launch_bounds__(W * 32, 1) few_up_kernel(const FewParams p) {
  using F = Fmt<WF>;
  constexpr int kThreads = W * 32;
  constexpr int kEntry = entry_bytes<WF>();
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  uint8_t* queue = smem + warp * (S * kEntry);
  float* part = reinterpret_cast<float*>(smem + W * S * kEntry);  // KS > 1: [2][warp][lane][4 NG]
  uint8_t* xs = reinterpret_cast<uint8_t*>(part + (KS > 1 ? 2 * kThreads * 4 * NG : 0));
  float* xf = reinterpret_cast<float*>(xs + p.T * p.x_ld);  // [T][ns] factors of x (kF16)
  const int ns = cdiv(p.H, F::kStepK);
  const Tables tb(reinterpret_cast<uint8_t*>(xf + (F::kF16 ? p.T * ns : 0)), p.T * p.k);
  pdl_wait();
  if (blockIdx.x == 0) {  // the tables are not there yet, before any CTA of the down kernel can look
    if (tid == 0) {
      *reinterpret_cast<volatile int32_t*>(p.tables + 4) = 0;
      __threadfence();
    }
    __syncthreads();
  }
  pdl_trigger();
  // x, with zeros up to a whole step
  const int xc = ns * (F::kStepK / 8);
  auto load_x = [&](int first, int n) {
    constexpr int kAt = F::kF16 ? 4 : 1;  // pieces of 8 values loaded before the first is worked on
    for (int i0 = first & ~31; i0 < p.T * xc; i0 += kAt * n) {
      uint4 raw[kAt];
      int tok[kAt], c[kAt];
#pragma unroll
      for (int j = 0; j < kAt; ++j) {
        const int i = i0 + j * n + lane;
        tok[j] = i / xc;
        c[j] = i - tok[j] * xc;
        const bool in = i < p.T * xc && c[j] * 8 < p.H;
        const uint16_t* src = p.x + (in ? (size_t)tok[j] * p.H + c[j] * 8 : 0);
        if constexpr (F::kF16) {
          raw[j] = make_uint4(0u, 0u, 0u, 0u);
          if (in) raw[j] = __ldcg(reinterpret_cast<const uint4*>(src));
        } else if (i < p.T * xc) {
          cp_async16_take(smem_u32(xs + tok[j] * p.x_ld + c[j] * 16), src, in);
        }
      }
      if constexpr (F::kF16) {
#pragma unroll
        for (int j = 0; j < kAt; ++j) {
          if (i0 + j * n >= p.T * xc) break;
          const uint32_t u[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
          float v[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[2 * e] = bf16_f32(u[e] & 0xFFFFu);
            v[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
          }
          uint4 o;
          const float f = f16_group<false>(v, o, o);
          if (tok[j] < p.T) {
            *reinterpret_cast<uint4*>(xs + tok[j] * p.x_ld + c[j] * 16) = o;
            if ((c[j] & 15) == 0) xf[tok[j] * ns + (c[j] >> 4)] = f;
          }
        }
      }
    }
  };
  const int nb = few_tables<NG>(p, tb, smem, blockIdx.x == 0, load_x);
  const int per = p.I / 8, units = nb * per;
  const int lo = (int)((int64_t)blockIdx.x * units / gridDim.x), hi = (int)((int64_t)(blockIdx.x + 1) * units / gridDim.x);
  const int row = p.H * F::kRowBytes / F::kStepK;  // bytes of a weight row
  constexpr int kNext = W / KS;  // to the team's next unit
  const int team = warp / KS, s0 = warp % KS;

  // A place in the warp's units: unit j, rows 8 r of block b
  struct Place {
    int j, b, r;
  };
  auto next = [&](Place& q) {
    q.j += kNext;
    q.r += kNext;
    while (q.r >= per) {
      q.r -= per;
      ++q.b;
    }
  };
  Place q{lo + team, 0, 0};
  q.b = q.j / per;
  q.r = q.j - q.b * per;

  // the next step to copy: step cs of place c, its weights for this lane at wp (gate) and
  // wp + up, its scales at sp
  Place c = q;
  int cs = s0, at = 0;
  const uint8_t *wp = p.pool, *sp = p.pool;
  const int64_t up = (int64_t)p.I * row;
  const int last = row % F::kRowBytes;  // bytes of a short last step
  auto set_rows = [&]() {
    if (c.j >= hi || s0 >= ns) return;
    const uint8_t* base = p.pool + (int64_t)tb.slot[c.b] * p.row_bytes;
    wp = base + (int64_t)(c.r * 8 + g) * row + 16 * t + s0 * F::kRowBytes;
    if constexpr (WF == OES_WFMT_FP8)
      sp = base + p.s13 + ((int64_t)((lane & 1) * cdiv(p.I, 128) + ((c.r * 8) >> 7)) * ns + s0) * 4;
    if constexpr (WF == OES_WFMT_NVFP4) {
      const int r16 = lane & 15;
      sp = base + p.s13 + ((int64_t)(2 * s0 + (lane >> 4)) * 2 * p.I + (r16 >> 3) * p.I + c.r * 8 + (r16 & 7)) * 4;
    }
  };
  set_rows();
  auto copy_next = [&]() {
    if (c.j < hi && s0 < ns) {
      const uint32_t e = smem_u32(queue + at * kEntry);
      const bool whole = last == 0 || cs + 1 < ns;
      if (whole) step_copy<WF>(e, wp, wp + up, 16, 16);
      else step_copy_last<WF>(e, wp, wp + up, 16, 16, last, p.pool);
      wp += KS * F::kRowBytes;
      if constexpr (WF == OES_WFMT_FP8) {
        if (lane < 2) cp_async4_take(e + 2048 + 4 * lane, sp, true);
        sp += 4 * KS;
      }
      if constexpr (WF == OES_WFMT_NVFP4) {
        const bool in = whole || lane < 16;
        cp_async4_take(e + 1024 + 4 * lane, in ? sp : p.pool, in);
        sp += (int64_t)16 * KS * p.I;
      }
      cs += KS;
      if (cs >= ns) {
        cs = s0;
        next(c);
        set_rows();
      }
    }
    cp_async_commit();
    at = at + 1 == S ? 0 : at + 1;
  };
#pragma unroll 1  // 8 tokens' FP8 time is 1 to 2 % longer with the copies written out
  for (int i = 0; i < S; ++i) copy_next();
  if (blockIdx.x == 0) {
    // the tables, for the down kernel
    few_order<NG>(p, tb, nb);
    if (tid == 0) *reinterpret_cast<int32_t*>(p.tables) = nb;
    for (int i = tid; i < down_tables_bytes(p.T * p.k) / 4; i += kThreads)
      reinterpret_cast<int32_t*>(p.tables + 16)[i] = reinterpret_cast<const int32_t*>(tb.w)[i];
    __syncthreads();
    if (tid == 0) {
      __threadfence();
      asm volatile("st.release.gpu.global.s32 [%0], 1;" ::"l"(p.tables + 4) : "memory");
    }
  }

  // columns past the tokens are not used: any row does
  uint32_t xb[NG], xfc[NG][2];
#pragma unroll
  for (int n = 0; n < NG; ++n) {
    xb[n] = smem_u32(xs + min(8 * n + g, p.T - 1) * p.x_ld) + 2 * piece_k<WF>(0, 0);
#pragma unroll
    for (int j = 0; j < 2; ++j) xfc[n][j] = smem_u32(xf + min(8 * n + 2 * t + j, p.T - 1) * ns);
  }
  int from = 0, buf = 0;
  // A unit for GN groups of eight tokens from n0 on.  Of more than eight tokens most blocks
  // have a route or two, in one group, and the other's instructions are left out.  (Here and
  // in a down kernel whose columns were tokens too: 16 tokens x 10 of 512 experts in bf16 228 -> 220
  // us, NVFP4 152 -> 144, 12 tokens 181 -> 173 and 124 -> 116.)
  auto unit = [&](auto groups, int n0) {
    constexpr int GN = decltype(groups)::value;
    uint32_t ub[GN], uf[GN][2];
#pragma unroll
    for (int n = 0; n < GN; ++n) {
      ub[n] = GN < NG && n0 > 0 ? xb[NG - 1] : xb[n];
#pragma unroll
      for (int j = 0; j < 2; ++j) uf[n][j] = GN < NG && n0 > 0 ? xfc[NG - 1][j] : xfc[n][j];
    }
    float acc[GN][4];
#pragma unroll
    for (int n = 0; n < GN; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
    float gs = 1.0f;  // needed at the end
    if constexpr (WF == OES_WFMT_NVFP4)
      gs = __ldcg(reinterpret_cast<const float*>(p.pool + (int64_t)tb.slot[q.b] * p.row_bytes + p.gs));
    for (int s = s0; s < ns; s += KS) {
      cp_async_wait<S - 1>();
      if (F::kScale) __syncwarp();  // scales that other lanes copied
      const uint32_t e = smem_u32(queue + from * kEntry);
      float d[GN][4], d1[GN][4];  // two chains of instructions with one group of tokens
      uint4 B[2][GN][F::kB];
#pragma unroll
      for (int hh = 0; hh < 2; ++hh)
#pragma unroll
        for (int n = 0; n < GN; ++n)
#pragma unroll
          for (int i = 0; i < F::kB; ++i)
            B[hh][n][i] = lds128(ub[n] + 2 * (s * F::kStepK + piece_k<WF>(hh, i) - piece_k<WF>(0, 0)));
      half_mma<WF, GN, true>(e, 0, B[0], d);
      if constexpr (GN == 1) {
        half_mma<WF, GN, true>(e, 1, B[1], d1);
#pragma unroll
        for (int i = 0; i < 4; ++i) d[0][i] += d1[0][i];
      } else {
        half_mma<WF, GN, false>(e, 1, B[1], d);
      }
      if constexpr (F::kF16) {
        float sg = 1.0f, su = 1.0f;
        if constexpr (WF == OES_WFMT_FP8) {
          const uint2 sc = lds64(e + 2048);
          sg = __uint_as_float(sc.x);
          su = __uint_as_float(sc.y);
        }
#pragma unroll
        for (int n = 0; n < GN; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float f = __uint_as_float(lds32(uf[n][j] + 4 * s));
            acc[n][j] = fmaf(sg * f, d[n][j], acc[n][j]);
            acc[n][2 + j] = fmaf(su * f, d[n][2 + j], acc[n][2 + j]);
          }
      } else {
#pragma unroll
        for (int n = 0; n < GN; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[n][i] += d[n][i];
      }
      if (F::kScale) __syncwarp();
      from = from + 1 == S ? 0 : from + 1;
      copy_next();
    }
    if constexpr (KS == 1) {
#pragma unroll
      for (int n = 0; n < GN; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = tb.route[q.b * 8 * NG + 8 * (n0 + n) + 2 * t + j];
          if (r >= 0) store_h<WF>(p, r, q.r * 8 + g, silu_f32(gs * acc[n][j]) * (gs * acc[n][2 + j]));
        }
    } else {
      float* mine = part + ((buf * W + warp) * 32 + lane) * (4 * NG);
#pragma unroll
      for (int n = 0; n < GN; ++n)
        *reinterpret_cast<float4*>(mine + 4 * n) =
            make_float4(gs * acc[n][0], gs * acc[n][1], gs * acc[n][2], gs * acc[n][3]);
      asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(KS * 32) : "memory");
      const int tt = tid - team * KS * 32;
      if (tt < 64 * GN) {
        const int col = tt >> 3, r8 = tt & 7, r = tb.route[q.b * 8 * NG + 8 * n0 + col];
        if (r >= 0) {
          const float* v = part + ((buf * W + team * KS) * 32 + r8 * 4 + (col & 7) / 2) * (4 * NG) + (col >> 3) * 4 + (col & 1);
          float gate = 0.0f, upv = 0.0f;
#pragma unroll
          for (int w = 0; w < KS; ++w) {
            gate += v[w * 32 * 4 * NG];
            upv += v[w * 32 * 4 * NG + 2];
          }
          store_h<WF>(p, r, q.r * 8 + r8, silu_f32(gate) * upv);
        }
      }
    }
  };
  for (; q.j < hi; next(q), buf ^= 1) {
    if constexpr (NG == 1) {
      unit(Int<1>{}, 0);
    } else {
      const uint32_t m = tb.has[q.b];
      if ((m & 0xFFu) && m >> 8) unit(Int<2>{}, 0);
      else unit(Int<1>{}, m >> 8 ? 1 : 0);
    }
  }
}

// ---------------------------------------------------------------------- down
// The (block, step of K) of a tile of rows are dealt out to the CTA's warps in runs.
// The rows of h of a step's tokens come through the warp's queue too, the first kRing of them
// (few blocks have more; those are loaded when they are needed).  For 8- and 4-bit weights they
// are fp32, and become pairs of f16 where they lie; for bf16 weights the first kernel left the three bf16
// numbers of each value (parted here, in every CTA, 16 tokens took 232 us where this takes 219).
// (Loaded by each lane as it needs them, their latency set the pace: 16 tokens
// x 10 of 200 bf16 experts ran at 1.9 TB/s.  Staged by the CTA for several blocks at a
// time, barriers and bookkeeping did.  With powers of two and pairs of f16 for each 8 values from the
// first kernel, one token of FP8 experts took 19 us, not 16.8.)
constexpr int kRing = 2;  // rows of h of a step in the queue

// A step of a row of h in shared memory, in kParts planes of 16-bit numbers: the three bf16 numbers of
// its values, or the two f16 numbers that the fp32 values become where they lie.  Pieces of 16 bytes
// have their places permuted (plane_at), so that the lanes that read a piece of neighbouring columns
// meet no bank twice.
template <int WF>
struct HRow {
  static constexpr int kParts = Fmt<WF>::kF16 ? 2 : 3, kPlane = Fmt<WF>::kStepK * 2;
  static constexpr int kRow = Fmt<WF>::kStepK * h_value_bytes(WF), kPieces = kRow / 16;  // also in memory
  static_assert(kRow == kParts * kPlane, "planes of a row");
};
// Piece c of plane `part` of a block's row r.
template <int WF>
__device__ __forceinline__ int plane_at(int r, int part, int c) {
  const int to = WF == OES_WFMT_BF16 ? c ^ 4 * ((r + part) & 1) : WF == OES_WFMT_FP8 ? c ^ part : c ^ c >> 3 ^ 2 * part;
  return part * HRow<WF>::kPlane + to * 16;
}
template <int WF, int S>
__host__ __device__ constexpr int down_queue_bytes() {  // and the rows of h in it
  return S * (entry_bytes<WF>() + kRing * HRow<WF>::kRow);
}
template <int WF, int NG, int S>
__host__ __device__ constexpr int down_warp_bytes() {  // queue, further rows (at a tile's end the sums), factors
  static_assert((8 * NG - kRing) * HRow<WF>::kRow >= 32 * 16 * NG, "a warp's sums");
  return down_queue_bytes<WF, S>() + (8 * NG - kRing) * HRow<WF>::kRow + (Fmt<WF>::kF16 ? 64 : 0);
}

// The columns of the instructions are the parts of a block's rows of h, row after row: a block of two
// routes in bf16, or of four in the other formats, fills one instruction's eight.  (With columns that belong to
// tokens and instructions of their own for the second parts, four tokens of NVFP4 experts took 42.4 us.)
template <int WF, int NG, int S>
__global__ void __launch_bounds__(W * 32, 1) few_down_kernel(const FewParams p) {
  using F = Fmt<WF>;
  using HR = HRow<WF>;
  constexpr int kThreads = W * 32, kParts = HR::kParts;
  constexpr int kEntry = entry_bytes<WF>(), kRow = HR::kRow;
  constexpr int kWarp = down_warp_bytes<WF, NG, S>();
  static_assert(kEntry % 64 == 0 && kWarp % 64 == 0 && (F::kF16 || (kEntry % 128 == 0 && kWarp % 128 == 0)), "permuted pieces");
  constexpr int kRowLanes = F::kStepK / 8, kRowsAt = 32 / kRowLanes;  // 8 values a lane: lanes a row, rows at a time
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  uint8_t* queue = smem + warp * kWarp;
  uint8_t* ring = queue + S * kEntry;                    // [S][kRing] rows of h
  uint8_t* more = ring + S * kRing * kRow;               // rows past those; at a tile's end [lane][4 NG] sums
  float* hf = reinterpret_cast<float*>(more + (8 * NG - kRing) * kRow);  // factors (kF16)
  const Tables tb(smem + W * kWarp, p.T * p.k);
  // The next kernel's CTAs take the SMs as this one's leave them (these fill an SM each) and wait
  // there for the last; left to the kernel's end, a call in a row takes 0.15 to 0.6 us more.
  pdl_trigger();
  // A CTA starts where one of few_up_kernel's has ended, some microseconds before all have
  // and what they wrote is sure to be seen.  The tables were written early and say
  // themselves that they are there; all else but h was complete before few_up_kernel passed its
  // own wait.  So where the tables are there (nothing waits for them), the queues are filled with
  // weights at once, and only h is waited for.
  __shared__ int s_early;
  if (tid == 0) {
    int f;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(f) : "l"(p.tables + 4) : "memory");
    s_early = f;
  }
  __syncthreads();
  const bool early = s_early == 1;
  if (!early) pdl_wait();
  // The tables as few_up_kernel left them.  A workspace that another call writes at the
  // same time would be a mistake of the caller's, which no address may follow: whatever
  // stands here, indexes are kept within their ranges.
  const int R = p.T * p.k, nb = min(max(__ldcg(reinterpret_cast<const int32_t*>(p.tables)), 0), R);
  for (int i = tid; i < down_tables_bytes(R) / 16; i += kThreads)
    reinterpret_cast<int4*>(tb.w)[i] = __ldcg(reinterpret_cast<const int4*>(p.tables + 16) + i);
  __syncthreads();
  for (int i = tid; i < nb; i += kThreads) {
    if ((uint32_t)tb.slot[i] >= (uint32_t)p.S) tb.slot[i] = 0;
    tb.has[i] &= (1u << p.T) - 1u;
    tb.cum[i] = (int16_t)min(max((int)tb.cum[i], 0), R - __popc(tb.has[i]));
  }
  for (int i = tid; i < R; i += kThreads)
    if ((uint32_t)tb.order[i] >= (uint32_t)R) tb.order[i] = 0;
  __syncthreads();
  const int row = p.I * F::kRowBytes / F::kStepK;
  const int ns = cdiv(p.I, F::kStepK);
  const int row_lo = blockIdx.x * p.rows_cta, row_hi = min(p.H, row_lo + p.rows_cta);

  // The warp's run of a tile: `run` (block, step of K), from block b0, step s0 on
  const int n_all = nb * ns, i0 = (int)((int64_t)warp * n_all / W);
  const int run = (int)((int64_t)(warp + 1) * n_all / W) - i0, b0 = i0 / ns, s0 = i0 - b0 * ns;

  // The next step to copy: step cs of block cb, `left` of the tile at row crow; its
  // weights for this lane at w0 and w1, its scales at sp, of its first rows of h at ho
  int cb = b0, cs = s0, left = run, crow = run > 0 ? row_lo : row_hi, at = 0;
  const uint8_t *w0 = p.pool, *w1 = p.pool, *sp = p.pool;
  int n0 = 0, n1 = 0;
  constexpr int kCopies = cdiv(kRing * HR::kPieces, 32);  // of 16 bytes a lane, for a step's rows of h
  int ho[kCopies];
  bool hin[kCopies];
  const int last = row % F::kRowBytes;  // bytes of a short last step
  bool sin = false;
  auto set_rows = [&]() {
    if (crow >= row_hi) return;
    const uint8_t* base = p.pool + (int64_t)tb.slot[cb] * p.row_bytes;
    // absent rows read nothing; any address in the pool stands in
    const bool ok0 = crow + g < row_hi, ok1 = crow + g + 8 < row_hi;
    const uint8_t* w = base + p.w2 + (int64_t)(crow + g) * row + cs * F::kRowBytes + 16 * t;
    w0 = ok0 ? w : p.pool;
    w1 = ok1 ? w + 8 * row : p.pool;
    n0 = ok0 ? 16 : 0;
    n1 = ok1 ? 16 : 0;
    if constexpr (WF == OES_WFMT_FP8) {
      const int r = crow + lane;
      sin = lane < kRowTile && r < row_hi;
      sp = sin ? base + p.s2 + ((int64_t)(r >> 7) * ns + cs) * 4 : p.pool;
    }
    if constexpr (WF == OES_WFMT_NVFP4) {
      const int r = crow + (lane & 15);
      sin = r < row_hi;
      sp = sin ? base + p.s2 + ((int64_t)(2 * cs + (lane >> 4)) * p.H + r) * 4 : p.pool;
    }
    const int first = tb.cum[cb], n = __popc(tb.has[cb]);
#pragma unroll
    for (int j = 0; j < kCopies; ++j) {
      const int pc = lane + 32 * j, rw = pc / HR::kPieces;
      hin[j] = rw < min(n, kRing);
      ho[j] = (hin[j] ? tb.order[first + rw] : 0) * p.I * h_value_bytes(WF) + cs * kRow + pc % HR::kPieces * 16;
    }
  };
  set_rows();
  auto piece_at = [&](int rw, int pc) {  // where a row's piece lies: fp32 as it comes, else in its plane
    return F::kF16 ? pc * 16 : plane_at<WF>(rw, pc / (HR::kPlane / 16), pc % (HR::kPlane / 16));
  };
  auto copy_h = [&](int slot, int j, int o) {  // o < 0: zeros
    const int pc = lane + 32 * j, rw = pc / HR::kPieces;
    if (pc < kRing * HR::kPieces)
      cp_async16_take(smem_u32(ring + (slot * kRing + rw) * kRow + piece_at(rw, pc % HR::kPieces)),
                      static_cast<const uint8_t*>(p.h) + max(o, 0), o >= 0);
  };
  auto copy_next = [&](int* later) {  // later: takes what copy_h is to be given
    if (crow < row_hi) {
      const uint32_t e = smem_u32(queue + at * kEntry);
      const bool whole = last == 0 || cs + 1 < ns;
      if (whole) step_copy<WF>(e, w0, w1, n0, n1);
      else step_copy_last<WF>(e, w0, w1, n0, n1, last, p.pool);
      w0 += F::kRowBytes;
      w1 += F::kRowBytes;
      if constexpr (WF == OES_WFMT_FP8) {
        if (lane < kRowTile) cp_async4_take(e + 2048 + 4 * lane, sp, sin);
        sp += 4;
      }
      if constexpr (WF == OES_WFMT_NVFP4) {
        const bool in = sin && (whole || lane < 16);
        cp_async4_take(e + 1024 + 4 * lane, in ? sp : p.pool, in);
        sp += sin ? (int64_t)8 * p.H : 0;
      }
#pragma unroll
      for (int j = 0; j < kCopies; ++j) {
        const int o = whole || cs * F::kStepK + lane * 4 < p.I ? ho[j] : -1;  // bf16's steps are whole
        if (later) later[j] = hin[j] ? o : -1;
        else if (hin[j]) copy_h(at, j, o);  // a row that the block has not is not read
        ho[j] += kRow;
      }
      const bool tile_done = --left == 0;
      if (++cs == ns || tile_done) {
        cs = tile_done ? s0 : 0;
        cb = tile_done ? b0 : cb + 1;
        if (tile_done) {
          left = run;
          crow += kRowTile;
        }
        set_rows();
      }
    }
    cp_async_commit();
    at = at + 1 == S ? 0 : at + 1;
  };
  {
    int later[S][kCopies];  // the first steps' rows of h
#pragma unroll
    for (int i = 0; i < S; ++i) {
#pragma unroll
      for (int j = 0; j < kCopies; ++j) later[i][j] = -1;
      copy_next(later[i]);
    }
    if (early) pdl_wait();  // h
#pragma unroll
    for (int i = 0; i < S; ++i) {
#pragma unroll
      for (int j = 0; j < kCopies; ++j) copy_h(i, j, later[i][j]);
      cp_async_commit();
    }
  }

  // The rows of h of a step of the block, n of them, `first` in the order.  For f16: 8 values of
  // row j to their parts in the row at `to`, those in the queue where they lie.
  const int hl = lane / kRowLanes, hp = lane % kRowLanes;
  auto form = [&](const float (&v)[8], uint8_t* to, int j, bool live) {
    uint4 x, y;
    const float f = f16_group<true>(v, x, y);
    if (live) {
      *reinterpret_cast<uint4*>(to + plane_at<WF>(j, 0, hp)) = x;
      *reinterpret_cast<uint4*>(to + plane_at<WF>(j, 1, hp)) = y;
      if (hp == 0) hf[j] = f;
    }
  };
  auto form_rows = [&](int first, int n, int step, int slot) {
    const uint8_t* h = static_cast<const uint8_t*>(p.h) + (int64_t)step * kRow;
    const int64_t ld = (int64_t)p.I * h_value_bytes(WF);
    if constexpr (F::kF16) {
      uint8_t* rows = ring + slot * kRing * kRow;
      float v[8];
      const float4* raw = reinterpret_cast<const float4*>(rows + min(hl, kRing - 1) * kRow + hp * 32);
      const float4 x = raw[0], y = raw[1];
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
      v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
      __syncwarp();  // read by all before it is written over
      form(v, rows + hl * kRow, hl, hl < kRing);
#pragma unroll 1
      for (int j = kRing; j < n; j += kRowsAt) {
        const bool live = j + hl < n;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.0f;
        if (live && step * F::kStepK + hp * 8 < p.I) {
          const float4* at = reinterpret_cast<const float4*>(h + tb.order[first + j + hl] * ld + hp * 32);
          const float4 a = __ldcg(at), b = __ldcg(at + 1);
          v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
          v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        }
        form(v, more + (j + hl - kRing) * kRow, j + hl, live);
      }
      __syncwarp();
    } else if (n > kRing) {
      // a piece of a row each for 24 lanes, four rows loaded together
      static_assert(F::kF16 || HR::kPieces <= 32, "bf16 rows of h");
      const bool on = lane < HR::kPieces;
      const uint32_t to = smem_u32(more) + piece_at(0, lane);
#pragma unroll 1
      for (int j0 = kRing; j0 < n; j0 += 4) {
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = make_uint4(0u, 0u, 0u, 0u);
          if (on && j0 + i < n) v[i] = __ldcg(reinterpret_cast<const uint4*>(h + tb.order[first + j0 + i] * ld + lane * 16));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)  // of row 1 the other half first, and so on
          if (on && j0 + i < n) sts128((to + (j0 + i - kRing) * kRow) ^ (i & 1 ? 64 : 0), v[i]);
      }
      __syncwarp();
    }
  };

  // The lane's operands of column v = 8 n + g: a block's parts lie plane after plane, the first
  // rows' in the queue and the others' behind it.  What lies there past the block's rows goes into
  // sums that are not used.
  constexpr int kPlane = HR::kPlane, kMost = cdiv(8 * NG * kParts, 8);  // instructions' columns
  const bool queued = g < kRing * kParts;
  const uint32_t swz = plane_at<WF>(g / kParts, g % kParts, piece_k<WF>(0, 0) / 8) - g % kParts * kPlane;
  const uint32_t hm = smem_u32(more) + (g - kRing * kParts) * kPlane + swz;
  const uint32_t h0 = queued ? smem_u32(ring) + g * kPlane + swz : hm, h0slot = queued ? kRing * kRow : 0;
  const uint32_t hfc = smem_u32(hf) + 4 * t;

  int from = 0;
  for (int row0 = row_lo; row0 < row_hi; row0 += kRowTile) {
    float acc[NG][4];  // of tokens 8 n + 2t and + 1, rows g and g + 8
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
#pragma unroll 1
    for (int b = b0, s1 = s0, rem = run; rem > 0; ++b) {
      const int end = min(ns, s1 + rem);
      rem -= end - s1;
      const uint32_t m = tb.has[b];
      const int first = tb.cum[b], n_rows = __popc(m), n8 = (n_rows * kParts + 7) / 8;
      constexpr int kSums = F::kF16 ? 2 : 4;  // f16: this lane's two columns are both parts of row 4 n + t, added at once
      float blk[kMost][kSums];
#pragma unroll
      for (int n = 0; n < kMost; ++n)
#pragma unroll
        for (int i = 0; i < kSums; ++i) blk[n][i] = 0.0f;
      float gs = 1.0f;  // needed at the end
      if constexpr (WF == OES_WFMT_NVFP4)
        gs = __ldcg(reinterpret_cast<const float*>(p.pool + (int64_t)tb.slot[b] * p.row_bytes + p.gs) + 1);
#pragma unroll 1
      for (int st = s1; st < end; ++st) {
        cp_async_wait<S - 1>();
        __syncwarp();  // what other lanes brought
        form_rows(first, n_rows, st, from);
        const uint32_t e = smem_u32(queue + from * kEntry);
        auto step = [&](auto groups) {  // GN instructions' columns
          constexpr int GN = decltype(groups)::value;
          float d[GN][4], d1[GN][4];  // two chains of instructions with one's columns
          uint4 B[2][GN][F::kB];
          auto load = [&](int hh) {
#pragma unroll
            for (int n = 0; n < GN; ++n)
#pragma unroll
              for (int i = 0; i < F::kB; ++i) {
                // the lane's pieces differ in these bits of their numbers, permuted or not
                constexpr int kHalf = WF == OES_WFMT_FP8 ? 0 : WF == OES_WFMT_BF16 ? 64 : 32;
                const uint32_t at = n == 0 ? h0 + from * h0slot : hm + n * (8 * kPlane);
                B[hh][n][i] = lds128((at ^ (kHalf * hh + 16 * i)) + (WF == OES_WFMT_FP8 ? 128 * hh : 0));
              }
          };
          load(0);
          if (GN <= 2) load(1);
          half_mma<WF, GN, true>(e, 0, B[0], d);
          if (GN > 2) load(1);
          if constexpr (GN == 1) {
            half_mma<WF, GN, true>(e, 1, B[1], d1);
#pragma unroll
            for (int i = 0; i < 4; ++i) d[0][i] += d1[0][i];
          } else {
            half_mma<WF, GN, false>(e, 1, B[1], d);
          }
          if constexpr (F::kF16) {
            float sc0 = 1.0f, sc1 = 1.0f;
            if constexpr (WF == OES_WFMT_FP8) {
              sc0 = __uint_as_float(lds32(e + 2048 + 4 * g));
              sc1 = __uint_as_float(lds32(e + 2048 + 32 + 4 * g));
            }
#pragma unroll
            for (int n = 0; n < GN; ++n) {
              const float f = __uint_as_float(lds32(hfc + 16 * n));
              blk[n][0] = fmaf(sc0 * f, d[n][0] + d[n][1], blk[n][0]);
              blk[n][1] = fmaf(sc1 * f, d[n][2] + d[n][3], blk[n][1]);
            }
          } else {
#pragma unroll
            for (int n = 0; n < GN; ++n)
#pragma unroll
              for (int i = 0; i < kSums; ++i) blk[n][i] += d[n][i];
          }
        };
        if (n8 <= 1) step(Int<1>{});
        else if (n8 == 2) step(Int<2>{});
        else if (NG == 2 && (F::kF16 || n8 > 3)) step(Int<kMost>{});
        else if constexpr (!F::kF16) step(Int<3>{});
        __syncwarp();  // read by all before the queue's entry is filled again
        from = from + 1 == S ? 0 : from + 1;
        copy_next(nullptr);
      }
      s1 = 0;
      // Each row's sums, its parts' columns together, to the lanes of its token, through the further
      // rows' place (by shuffles, row after row, whose code is fetched anew each time, 16 tokens x 10 of 32
      // bf16 experts took 82 us, so 79).  A token without a route in this block takes nothing from it, not
      // even a NaN of its weights.
      constexpr int kCols = F::kF16 ? 4 * kMost : 8 * kMost, kLd = kCols + 4;  // a row's sums; of each of 16 rows of out
      static_assert((8 * NG - kRing) * kRow >= 16 * kLd * 4, "a block's sums");
      float* sums = reinterpret_cast<float*>(more);
#pragma unroll
      for (int n = 0; n < kMost; ++n)
        if (n < n8) {
          if constexpr (F::kF16) {
            sums[g * kLd + 4 * n + t] = blk[n][0];
            sums[(g + 8) * kLd + 4 * n + t] = blk[n][1];
          } else {
            *reinterpret_cast<float2*>(sums + g * kLd + 8 * n + 2 * t) = make_float2(blk[n][0], blk[n][1]);
            *reinterpret_cast<float2*>(sums + (g + 8) * kLd + 8 * n + 2 * t) = make_float2(blk[n][2], blk[n][3]);
          }
        }
      __syncwarp();
#pragma unroll
      for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int col = 8 * n + 2 * t + j;
          if ((m >> col) & 1u) {
            const int r = __popc(m & ((1u << col) - 1));
            const float f = tb.w[tb.order[first + r]] * gs;
            constexpr int kEach = F::kF16 ? 1 : kParts;
            const float* v = sums + g * kLd + r * kEach;
            float sum0 = v[0], sum1 = v[8 * kLd];
#pragma unroll
            for (int part = 1; part < kEach; ++part) {
              sum0 += v[part];
              sum1 += v[8 * kLd + part];
            }
            acc[n][j] = fmaf(f, sum0, acc[n][j]);
            acc[n][2 + j] = fmaf(f, sum1, acc[n][2 + j]);
          }
        }
      __syncwarp();  // read before others' sums or rows come there
    }
    float* mine = reinterpret_cast<float*>(more) + lane * (4 * NG);
#pragma unroll
    for (int n = 0; n < NG; ++n)
      *reinterpret_cast<float4*>(mine + 4 * n) = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
    __syncthreads();
    for (int i = tid; i < kRowTile * p.T; i += kThreads) {
      const int r16 = i & 15, tok = i >> 4;
      if (row0 + r16 >= row_hi) continue;
      const float* v = reinterpret_cast<const float*>(smem + down_queue_bytes<WF, S>()) +
                       ((r16 & 7) * 4 + (tok & 7) / 2) * (4 * NG) + (tok >> 3) * 4 + (r16 >> 3) * 2 + (tok & 1);
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += v[w * (kWarp / 4)];
      p.out[(int64_t)tok * p.H + row0 + r16] = (uint16_t)f32_bf16(s);
    }
    if (row0 + kRowTile < row_hi) __syncthreads();  // read before the next tile's rows of h come there
  }
}

// ------------------------------------------------------------------ launches
constexpr size_t kSmemMost = 227 * 1024 - 5 * 1024;  // beside the kernels' static shared memory

template <int WF>
int x_stride(int H) {
  using F = Fmt<WF>;
  // rows a bank's width apart, so that the eight lanes of a phase never meet
  return ceil_div(H, F::kStepK) * F::kStepK * 2 + F::kXPad;
}

template <int WF, int NG, int KS, int S>
size_t up_smem(int T, int k, int H) {
  using F = Fmt<WF>;
  return (size_t)W * S * entry_bytes<WF>() + (KS > 1 ? 2 * W * 32 * 16 * NG : 0) + (size_t)T * x_stride<WF>(H) +
         (F::kF16 ? 4 * T * ceil_div(H, F::kStepK) : 0) + tables_bytes(T * k, NG);
}

template <int WF, int NG, int KS, int S>
int launch_up(const FewParams& p, cudaStream_t stream) {
  const size_t smem = up_smem<WF, NG, KS, S>(p.T, p.k, p.H);
  int rc = set_max_dynamic_smem(reinterpret_cast<const void*>(few_up_kernel<WF, NG, KS, S>), smem,
                                "few_up_kernel: shared memory limit");
  if (rc) return rc;
  const int64_t units = (int64_t)p.T * p.k * (p.I / 8);  // at most
  launch_kernel(few_up_kernel<WF, NG, KS, S>, (int)std::min<int64_t>(num_sms(), units), W * 32, smem, stream, p);
  OES_CHECK_LAUNCH("few_up_kernel");
  return OES_OK;
}

constexpr size_t kDownSmemMost = 227 * 1024 - 128;  // few_down's own, beside its static shared memory
template <int WF, int NG, int S>
constexpr size_t down_smem(int T, int k) {
  return (size_t)W * down_warp_bytes<WF, NG, S>() + down_tables_bytes(T * k);
}
template <int WF, int NG, int S>
int launch_down(const FewParams& p, cudaStream_t stream) {
  static_assert(down_smem<WF, NG, S>(8 * NG, OES_MAX_TOPK) <= kDownSmemMost, "few_down's shared memory");
  const size_t smem = down_smem<WF, NG, S>(p.T, p.k);
  int rc = set_max_dynamic_smem(reinterpret_cast<const void*>(few_down_kernel<WF, NG, S>), smem,
                                      "few_down_kernel: shared memory limit");
  if (rc) return rc;
  launch_kernel(few_down_kernel<WF, NG, S>, ceil_div(p.H, p.rows_cta), W * 32, smem, stream, p);
  OES_CHECK_LAUNCH("few_down_kernel");
  return OES_OK;
}

// One group of tokens: both kernels.
template <int WF, int NG>
int launch_few(FewParams p, cudaStream_t stream) {
  p.x_ld = x_stride<WF>(p.H);
  p.rows_cta = ceil_div(p.H, num_sms());
  // Warps a unit: one of a CTA's sixteen keeps 8 KB in flight, so that few units on an
  // SM do not fill it.  Up to two units an SM: 1 token x 2 experts of 2048 x 128, bf16,
  // takes 8.7 us with 16 warps a unit and 11.8 with one, 1 x 1 of 4096 x 512 10.7 and
  // 17.1; up to eight: 1 x 10 of 2048 x 768 24.4 us with 4 and 25.1 with one (with 16,
  // in FP8, 19.3 against 17.3).
  const int64_t units = (int64_t)p.T * p.k * (p.I / 8);  // at most
  const auto fits = [&](size_t smem) { return smem <= kSmemMost; };
  int rc;
  if (units <= 2 * num_sms() && fits(up_smem<WF, NG, 16, 2>(p.T, p.k, p.H))) rc = launch_up<WF, NG, 16, 2>(p, stream);
  else if (units <= 8 * num_sms() && fits(up_smem<WF, NG, 4, 3>(p.T, p.k, p.H))) rc = launch_up<WF, NG, 4, 3>(p, stream);
  else if (fits(up_smem<WF, NG, 1, 4>(p.T, p.k, p.H))) rc = launch_up<WF, NG, 1, 4>(p, stream);
  else rc = launch_up<WF, NG, 1, 2>(p, stream);
  if (rc) return rc;
  // Three steps in the second kernel's queues; those of FP8 experts do not fit for more than
  // eight tokens.
  return launch_down<WF, NG, WF == OES_WFMT_FP8 && NG == 2 ? 2 : 3>(p, stream);
}

// Most tokens whose rows of x fit beside the shortest queues.
template <int WF>
int group_tokens(int T, int k, int H) {
  int n = T;
  while (n > 1 && (n > 8 ? up_smem<WF, 2, 1, 2>(n, k, H) : up_smem<WF, 1, 1, 2>(n, k, H)) > kSmemMost) --n;
  return n;
}

template <int WF>
int run_few(FewParams p, cudaStream_t stream) {
  const int T = p.T, groups = ceil_div(T, group_tokens<WF>(T, p.k, p.H)), per = ceil_div(T, groups);
  for (int t0 = 0; t0 < T; t0 += per) {
    FewParams q = p;
    q.T = std::min(per, T - t0);
    q.x += (size_t)t0 * p.H;
    q.out += (size_t)t0 * p.H;
    q.ids += (size_t)t0 * p.k;
    q.weights += (size_t)t0 * p.k;
    if (p.logits) q.logits = static_cast<const uint8_t*>(p.logits) + (size_t)t0 * p.E * (p.logits_bf16 ? 2 : 4);
    const int rc = q.T > 8 ? launch_few<WF, 2>(q, stream) : launch_few<WF, 1>(q, stream);
    if (rc) return rc;
  }
  return OES_OK;
}

}  // namespace
}  // namespace oes

using namespace oes;

namespace {
// The view's own limits; shared by the size query and the call.
int check_view(const oes_routed_experts* v, int T, int k, const char* who) {
  OES_REQUIRE(v, "%s: null view", who);
  OES_REQUIRE(v->E >= 1 && v->E <= OES_MAX_EXPERTS && v->S >= 1, "%s: bad E=%d S=%d", who, v->E, v->S);
  OES_REQUIRE(v->H >= 64 && v->I >= 64 && v->H % 64 == 0 && v->I % 64 == 0 && v->H <= 16384 && v->I <= 16384,
              "%s: H=%d I=%d must be multiples of 64 in [64, 16384]", who, v->H, v->I);
  OES_REQUIRE(v->wfmt >= OES_WFMT_BF16 && v->wfmt <= OES_WFMT_FP8, "%s: bad wfmt %d", who, v->wfmt);
  OES_REQUIRE(T >= 0 && k >= 1 && k <= OES_MAX_TOPK, "%s: bad T=%d k=%d", who, T, k);
  if (v->wfmt == OES_WFMT_NVFP4_W4A4) {
    set_error("%s: activations are not quantised here (OES_WFMT_NVFP4 reads the same rows)", who);
    return OES_ERR_UNSUPPORTED;
  }
  if (T > OES_FEW_TOKENS_MAX) {
    set_error("%s: %d tokens, at most %d", who, T, OES_FEW_TOKENS_MAX);
    return OES_ERR_UNSUPPORTED;
  }
  return OES_OK;
}
static_assert(OES_FEW_TOKENS_MAX == kMaxTokens, "tokens a call");
}  // namespace

extern "C" size_t moe_layer_few_tokens_workspace_size(const oes_routed_experts* v, int T, int k) {
  if (check_view(v, T, k, "moe_layer_few_tokens_workspace_size") || T == 0) return 0;
  // h, then the tables of a group of tokens
  return ((size_t)T * k * v->I * h_value_bytes(v->wfmt) + 16 + down_tables_bytes(T * k) + 255) / 256 * 256;
}

extern "C" int moe_layer_few_tokens(const oes_routed_experts* v, const uint16_t* x, int T, int k, const void* logits,
                                    int dtype, int32_t* ids, float* weights, void* workspace, size_t workspace_bytes,
                                    uint16_t* out, int32_t* status, oes_stream_t stream) {
  const char* who = "moe_layer_few_tokens";
  int rc = check_view(v, T, k, who);
  if (rc) return rc;
  OES_REQUIRE(dtype == OES_LOGITS_F32 || dtype == OES_LOGITS_BF16, "%s: unknown logits type %d", who, dtype);
  OES_REQUIRE(!logits || k <= v->E, "%s: k=%d of E=%d experts", who, k, v->E);
  if (T == 0) return OES_OK;
  OES_REQUIRE(v->pool && v->e2s && x && ids && weights && workspace && out, "%s: null pointer", who);
  const Fp8Row f8 = fp8_row(v->H, v->I);
  const int64_t hi = (int64_t)v->H * v->I;
  FewParams p{};
  int64_t need;
  if (v->wfmt == OES_WFMT_BF16) {
    p.w2 = 4 * hi;
    need = 6 * hi;
  } else if (v->wfmt == OES_WFMT_FP8) {
    p.s13 = f8.s13;
    p.w2 = f8.w2;
    p.s2 = f8.s2;
    need = f8.end;
  } else {
    p.s13 = hi;
    p.w2 = p.s13 + hi / 8;
    p.s2 = p.w2 + hi / 2;
    p.gs = p.s2 + hi / 16;
    need = p.gs + 16;
  }
  OES_REQUIRE(v->row_bytes >= need && v->row_bytes % 16 == 0, "%s: row_bytes %lld (layout needs %lld, multiple of 16)",
              who, (long long)v->row_bytes, (long long)need);
  OES_REQUIRE(((uintptr_t)v->pool & 15) == 0 && ((uintptr_t)x & 15) == 0 && ((uintptr_t)workspace & 15) == 0,
              "%s: pool, x and workspace must be 16-byte aligned", who);
  OES_REQUIRE((((uintptr_t)ids | (uintptr_t)weights | (uintptr_t)v->e2s | (uintptr_t)status) & 3) == 0 &&
                  ((uintptr_t)out & 1) == 0 && ((uintptr_t)logits & (dtype == OES_LOGITS_F32 ? 3 : 1)) == 0,
              "%s: a pointer is not aligned to its type", who);
  const size_t bytes = moe_layer_few_tokens_workspace_size(v, T, k);
  OES_REQUIRE(workspace_bytes >= bytes, "%s: workspace %zu < %zu bytes", who, workspace_bytes, bytes);
  p.pool = static_cast<const uint8_t*>(v->pool);
  p.row_bytes = v->row_bytes;
  p.e2s = v->e2s;
  p.E = v->E;
  p.S = v->S;
  p.H = v->H;
  p.I = v->I;
  p.T = T;
  p.k = k;
  p.x = x;
  p.logits = logits;
  p.logits_bf16 = dtype == OES_LOGITS_BF16;
  p.ids = ids;
  p.weights = weights;
  p.h = workspace;
  p.tables = static_cast<uint8_t*>(workspace) + (size_t)T * k * v->I * h_value_bytes(v->wfmt);
  p.out = out;
  p.status = status;
  if (logits && v->E > kFusedExperts) {
    // wider rows are routed by the router's own kernel: held 16 a lane, a row of 512
    // fits these kernels' registers
    if ((rc = moe_route_topk(logits, dtype, T, v->E, k, ids, weights, stream))) return rc;
    p.logits = nullptr;
  }
  if (v->wfmt == OES_WFMT_BF16) return run_few<OES_WFMT_BF16>(p, stream);
  if (v->wfmt == OES_WFMT_FP8) return run_few<OES_WFMT_FP8>(p, stream);
  return run_few<OES_WFMT_NVFP4>(p, stream);
}
