// The units of work of the grouped GEMM kernels: one (align block, weight tile)
// pair each, looked up in the routing tables and dealt out to the CTAs.
#pragma once

#include "common.cuh"
#include "gemm_types.h"

namespace oes {

constexpr int kTileM = 128;           // weight rows per MMA (weight-major kernels)
constexpr int kMaxUnitsPerCta = 256;  // units whose info is tabled in shared memory

struct Unit {
  int b, m, h, slot, nvalid;  // h: the unit's K half (0 unless the tile's K is split)
  bool skip;
};

constexpr int kFiltered = -2;  // Unit::slot of a block another launch computes

// A routing-table entry: through L2 alone (ld.global.cg) for a kernel that
// reads the tables before its dependency wait (GEMM2, see the kernel), else
// a plain load.
template <bool CG>
__device__ __forceinline__ int32_t ld_tab(const int32_t* p) { return CG ? __ldcg(p) : *p; }
template <bool CG>
__device__ __forceinline__ int32_t ld_tab(const uint8_t* p) { return CG ? __ldcg(p) : *p; }

// Number of routes of block b (padding, value R, only at its end).
template <bool CG>
__device__ __forceinline__ int block_nvalid(const GemmParams& p, int b) {
  const int32_t* s = p.sorted_ids + (int64_t)b * p.BN;
  if (ld_tab<CG>(s + p.BN - 1) < p.R) return p.BN;
  int lo = 0, hi = p.BN - 1;  // first index holding padding
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ld_tab<CG>(s + mid) < p.R) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// The same for blocks of 16 to 128 (a multiple of 16), in two rounds of
// independent loads (one for 16) where the search takes one load after another.
// An FP8 layer's call for one token took 28.0 us so, 29.2 with the search.
template <bool CG>
__device__ __forceinline__ int block_nvalid_wide(const GemmParams& p, int b) {
  const int32_t* s = p.sorted_ids + (int64_t)b * p.BN;
  const int parts = p.BN >> 4;
  int full = 0, n = 0;
  if (parts > 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) full += i < parts && ld_tab<CG>(s + 16 * i + 15) < p.R;
    if (full == parts) return p.BN;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) n += ld_tab<CG>(s + 16 * full + i) < p.R;
  return 16 * full + n;
}

// Which block / tile a unit is, the slot of its expert, and how many of the
// block's entries are real routes (padding, value R, only at the end).
template <bool CG, bool WIDE = false>
__device__ __forceinline__ Unit unit_info(const GemmParams& p, int u, int nb) {
  // tile index fastest (after the K half): the units of one block run on
  // neighbouring CTAs at the same time, so the block's token rows (GEMM1) or
  // h rows (GEMM2) are read from DRAM once and then served from L2 for its
  // other tiles
  Unit t;
  const int upb = p.n_mtiles * p.ks;  // units per block
  t.b = u / upb;
  t.m = (u % upb) / p.ks;
  t.h = (u % upb) % p.ks;
  const int e = ld_tab<CG>(p.block_expert + t.b);
  if (WIDE) t.nvalid = block_nvalid_wide<CG>(p, t.b);
  const bool valid_e = e >= 0 && e < p.E;
  const bool filtered = p.filter && valid_e && ld_tab<CG>(p.flags + e) != p.filter;
  t.slot = filtered ? kFiltered : (valid_e ? ld_tab<CG>(p.e2s + e) : -1);
  if (!WIDE) t.nvalid = block_nvalid<CG>(p, t.b);
  t.skip = t.slot < 0 || t.slot >= p.S || t.nvalid == 0;
  return t;
}

__device__ __forceinline__ int round16(int n) { return (n + 15) & ~15; }

// K chunks [kc_lo, kc_hi) of a unit: all of the tile's, or those of its half
__device__ __forceinline__ int kc_lo(const GemmParams& p, const Unit& t) { return t.h * p.n_kc / p.ks; }
__device__ __forceinline__ int kc_hi(const GemmParams& p, const Unit& t) {
  return (t.h + 1) * p.n_kc / p.ks;
}

struct UnitRec {  // shared-memory copy of a Unit; m holds tile * ks + K half
  int b, m, slot, nvalid;
};


// A filtered launch deals out only the units of the selected blocks, densely,
// so that its CTAs get equal shares: the selected block of rank g (blocks in
// order) owns units g * upb + m, upb = n_mtiles * ks (tile fastest after the
// K half, as everywhere), and this
// worker (a CTA, or the CTAs of a cluster) takes every nworkers-th of them into
// its table.  Every CTA computes the same ranks.  Returns the number of units, or -1 when this CTA's share would
// not fit the table (the caller then numbers units as an unfiltered launch and
// skips the filtered ones).  All threads of the CTA call it.
template <bool CG>
__device__ __forceinline__ int fill_filtered_units(const GemmParams& p, int nb, UnitRec* utab, int* s_scan,
                                   int worker, int nworkers) {
  const int tid = threadIdx.x, nthr = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int nw = nthr >> 5;
  auto selected = [&](int b) {
    const int e = ld_tab<CG>(p.block_expert + b);
    return e >= 0 && e < p.E && ld_tab<CG>(p.flags + e) == p.filter &&
           ld_tab<CG>(p.sorted_ids + (int64_t)b * p.BN) < p.R;
  };
  if (nb <= nthr) {
    // one block per thread: its expert and its ids, then the expert's group
    // and slot, two rounds of independent loads
    bool sel = false;
    int nvalid = 0, slot = -1;
    if (tid < nb) {
      const int e = ld_tab<CG>(p.block_expert + tid);
      nvalid = block_nvalid<CG>(p, tid);
      if (e >= 0 && e < p.E) {
        const int f = ld_tab<CG>(p.flags + e);
        slot = ld_tab<CG>(p.e2s + e);
        sel = f == p.filter && nvalid > 0;
      }
    }
    const unsigned bal = __ballot_sync(0xffffffffu, sel);
    if (lane == 0) s_scan[warp] = __popc(bal);
    __syncthreads();
    int off = 0, n = 0;
    for (int i = 0; i < nw; ++i) {
      if (i < warp) off += s_scan[i];
      n += s_scan[i];
    }
    const int upb = p.n_mtiles * p.ks;
    const int units = n * upb;
    if (units > kMaxUnitsPerCta * nworkers) return -1;
    if (sel) {
      const int g = off + __popc(bal & ((1u << lane) - 1u));
      for (int m = 0; m < upb; ++m) {
        const int v = g * upb + m;
        if (v % nworkers == worker) utab[v / nworkers] = UnitRec{tid, m, slot, nvalid};
      }
    }
    return units;
  }
  int mine = 0;
  for (int b = tid; b < nb; b += nthr) mine += selected(b) ? 1 : 0;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) s_scan[warp] = mine;
  __syncthreads();
  if (tid == 0) {
    int n = 0;
    for (int i = 0; i < nw; ++i) n += s_scan[i];
    s_scan[32] = n;
  }
  __syncthreads();
  const int upb = p.n_mtiles * p.ks;
  const int units = s_scan[32] * upb;
  __syncthreads();
  if (units > kMaxUnitsPerCta * nworkers) return -1;
  int base = 0;
  for (int b0 = 0; b0 < nb; b0 += nthr) {
    const int b = b0 + tid;
    const bool sel = b < nb && selected(b);
    const unsigned bal = __ballot_sync(0xffffffffu, sel);
    if (lane == 0) s_scan[warp] = __popc(bal);
    __syncthreads();
    int off = base, chunk = 0;
    for (int i = 0; i < nw; ++i) {
      if (i < warp) off += s_scan[i];
      chunk += s_scan[i];
    }
    if (sel) {
      const int g = off + __popc(bal & ((1u << lane) - 1u));
      const int nvalid = block_nvalid<CG>(p, b);
      const int slot = ld_tab<CG>(p.e2s + ld_tab<CG>(p.block_expert + b));
      for (int m = 0; m < upb; ++m) {
        const int v = g * upb + m;
        if (v % nworkers == worker) utab[v / nworkers] = UnitRec{b, m, slot, nvalid};
      }
    }
    base += chunk;
    __syncthreads();
  }
  return units;
}

// The CTA's u-th unit (u counted in this CTA's sequence), from the table
// filled at kernel start, or computed directly past the table's end.
template <bool CG>
__device__ __forceinline__ Unit my_unit(const GemmParams& p, const UnitRec* tab, int idx, int u, int nb) {
  if (idx < kMaxUnitsPerCta) {
    const UnitRec r = tab[idx];
    Unit t;
    t.b = r.b;
    t.m = r.m / p.ks;
    t.h = r.m % p.ks;
    t.slot = r.slot;
    t.nvalid = r.nvalid;
    t.skip = t.slot < 0 || t.slot >= p.S || t.nvalid == 0;
    return t;
  }
  return unit_info<CG>(p, u, nb);
}

}  // namespace oes
