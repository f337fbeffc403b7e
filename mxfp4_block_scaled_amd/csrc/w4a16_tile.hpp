// Arguments and a wave's work lookup of the FP4-weight x bf16-activation kernels over ragged rows
// (w4a16_tile_body.hpp, w4a16_tile.hip, w4a16_grouped.hip, w4a16_lora.hip).
#pragma once

#include "w4a16_common.hpp"
#include "w4a16_plan.hpp"

namespace mxf {

struct W16TileArgs {
  const uint16_t* a;       // [a_rows][K] bf16
  int64_t a_rows;
  const int32_t* offsets;  // grouped: [E+1] row ranges of the experts; null: rows [0, R) of one matrix
  const int32_t* pair;     // null: row r reads a's row r; else a's row pair[r] / topk
  int topk, E;
  int min_rows, max_rows;  // grouped: only experts of min_rows < rows <= max_rows
  int64_t R;               // rows of out
  const uint8_t* w;        // [E][N][K/2] codes
  const uint8_t* ws;       // [E][N][K/32] UE8M0 or [E][N][K/16] UE4M3
  int64_t N, K;
  void* out;               // [R][N] or, with SwiGLU, [R][N/2]
  int ntiles;
  // adapters (w4a16_lora.hip)
  const float* low;         // [lslices][R][rank]: scaling * a . lora_a^T, K slice by K slice
  int rank, L, S, lslices;
  int kslices;              // K slices of a sliced product
  const int32_t* seg_off;      // [S+1]
  const int32_t* seg_adapter;  // [S]
  const uint16_t* lora_b;      // [L][N][rank] bf16
};

// Item j of XCD x: the units' items are split into 8 contiguous ranges, one per XCD, so that the
// workgroups of an XCD share activation rows and weight tiles in its L2. Called by whole waves;
// false: none. Every workgroup starts with this, so its latency counts (w16_lane_units).
template <int BM, int CE>
__device__ __forceinline__ bool w16_item_of(const int32_t* __restrict__ off, int E, int64_t R, int lo_rows, int hi_rows,
                                            int ntiles, int x, int j, int& e_out, int& n_out, int64_t& row0, int& m) {
  const int lane = threadIdx.x & 63;
  int o[CE + 1];
  const int units = w16_lane_units<BM, CE>(off, E, R, lo_rows, hi_rows, lane, o);
  int incl = units;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(incl, d);
    if (lane >= d) incl += y;
  }
  const int excl = incl - units;
  // the host keeps units x ntiles below 2^31
  const uint32_t total = (uint32_t)__builtin_amdgcn_readlane(incl, 63) * (uint32_t)ntiles;
  uint32_t w;
  if (!w16_range(total, x, j, w)) return false;
  const int p = (int)(w / (uint32_t)ntiles);
  const bool mine = p >= excl && p < incl;
  const unsigned long long msk = __ballot(mine);
  if (msk == 0) return false;
  const int src = __ffsll((long long)msk) - 1;
  W16Pick k{0, 0, 1, 0, 0};
  if (mine) k = w16_lane_find<BM, CE>(off, E, R, lo_rows, hi_rows, lane, o, excl, p);
  k.e = __builtin_amdgcn_readlane(k.e, src);
  k.before = __builtin_amdgcn_readlane(k.before, src);
  k.units = __builtin_amdgcn_readlane(k.units, src);
  k.rows = __builtin_amdgcn_readlane(k.rows, src);
  k.row0 = __builtin_amdgcn_readlane(k.row0, src);
  e_out = k.e;
  return w16_item_place<BM>(k, w, ntiles, n_out, row0, m);
}

template <int BM>
__device__ __forceinline__ bool w16_item(const int32_t* __restrict__ off, int E, int64_t R, int lo_rows, int hi_rows,
                                         int ntiles, int x, int j, int& e_out, int& n_out, int64_t& row0, int& m) {
  if (E <= 64) return w16_item_of<BM, 1>(off, E, R, lo_rows, hi_rows, ntiles, x, j, e_out, n_out, row0, m);
  if (E <= 256) return w16_item_of<BM, 4>(off, E, R, lo_rows, hi_rows, ntiles, x, j, e_out, n_out, row0, m);
  return w16_item_of<BM, 0>(off, E, R, lo_rows, hi_rows, ntiles, x, j, e_out, n_out, row0, m);
}

// first segment s whose end seg_off[s + 1] lies past row t (S if none): 64 probes a step
__device__ __forceinline__ int first_segment(const int32_t* __restrict__ seg_off, int S, int64_t t) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = S;
  while (lo < hi) {
    const bool one = w16_probe_step(lo, hi) == 1;
    w16_probe_narrow(__ballot(w16_probe(seg_off, lo, hi, lane, t)), lo, hi);
    if (one) break;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

void launch_w16_tile_grouped(const W16TileArgs& a, bool nv, bool swiglu, bool out_bf16, const W16Launch& l,
                             hipStream_t stream);
void launch_w16_tile_lora(const W16TileArgs& a, bool nv, bool out_bf16, const W16LoraPlan& l, hipStream_t stream);

}  // namespace mxf
