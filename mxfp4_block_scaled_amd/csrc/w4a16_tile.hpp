// Arguments and work lookup of the FP4-weight x bf16-activation kernels over ragged rows
// (w4a16_tile.hip, w4a16_grouped.hip, w4a16_lora.hip).
#pragma once

#include "w4a16_common.hpp"

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
  const float* low;        // [nslice][R][rank] fp32, the slices' sum is scaling * a . lora_a^T
  int nslice, rank, L, S;
  const int32_t* seg_off;      // [S+1]
  const int32_t* seg_adapter;  // [S]
  const uint16_t* lora_b;      // [L][N][rank] bf16
};

// Rows of expert e as stored, held inside [0, R): offsets that are not ascending or leave
// the range cannot lead outside the operands.
__device__ __forceinline__ int w16_rows(const int32_t* __restrict__ off, int64_t R, int e, int64_t& lo) {
  lo = min(max((int64_t)off[e], (int64_t)0), R);
  const int64_t hi = min(max((int64_t)off[e + 1], lo), R);
  return (int)(hi - lo);
}

// Units of an expert of c rows in a launch for experts of lo_rows < c <= hi_rows:
// ceil(c / BM), or one when BM == 0.
template <int BM>
__device__ __forceinline__ int w16_units(int c, int lo_rows, int hi_rows) {
  if (c <= lo_rows || c > hi_rows) return 0;
  if constexpr (BM == 0) return 1;
  else return (c + BM - 1) / BM;
}

// Item j of XCD x: the units' items (n-tile by n-tile inside an expert, unit by unit inside
// an n-tile) are split into 8 contiguous ranges, one per XCD, so that the workgroups of an
// XCD share activation rows and weight tiles in its L2. Called by whole waves; false: none.
template <int BM>
__device__ __forceinline__ bool w16_item(const int32_t* __restrict__ off, int E, int64_t R, int lo_rows, int hi_rows,
                                         int ntiles, int x, int j, int& e_out, int& n_out, int64_t& row0, int& m) {
  const int lane = threadIdx.x & 63;
  const int C = (E + 63) >> 6, first = lane * C;
  int units = 0;
  int64_t r0;
  for (int i = 0; i < C; ++i)
    if (first + i < E) units += w16_units<BM>(w16_rows(off, R, first + i, r0), lo_rows, hi_rows);
  int incl = units;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(incl, d);
    if (lane >= d) incl += y;
  }
  const int excl = incl - units;
  const int64_t total = (int64_t)__shfl(incl, 63) * ntiles;
  const int64_t w = x * total / 8 + j;
  if (w >= (x + 1) * total / 8) return false;
  const int p = (int)(w / ntiles);
  const bool mine = p >= excl && p < incl;
  const unsigned long long msk = __ballot(mine);
  if (msk == 0) return false;
  const int src = __ffsll((long long)msk) - 1;
  int ee = 0, ue = 0, ke = 1;
  if (mine) {
    int acc = excl;
    for (int i = 0; i < C && first + i < E; ++i) {
      const int n = w16_units<BM>(w16_rows(off, R, first + i, r0), lo_rows, hi_rows);
      if (p < acc + n) {
        ee = first + i;
        ue = acc;
        ke = n;
        break;
      }
      acc += n;
    }
  }
  ee = __builtin_amdgcn_readfirstlane(__shfl(ee, src));
  ue = __shfl(ue, src);
  ke = __shfl(ke, src);
  const int64_t local = w - (int64_t)ue * ntiles;
  n_out = __builtin_amdgcn_readfirstlane((int)(local / ke));
  const int loc = __builtin_amdgcn_readfirstlane((int)(local % ke));
  if (n_out < 0 || n_out >= ntiles || loc < 0) return false;
  e_out = ee;
  const int c = w16_rows(off, R, ee, r0);
  row0 = r0 + (int64_t)loc * BM;
  m = BM == 0 ? c : min(BM, c - loc * BM);
  return m > 0;
}

void launch_w16_tile_grouped(const W16TileArgs& a, bool nv, bool swiglu, bool out_bf16, int bm, int64_t units,
                             hipStream_t stream);
void launch_w16_tile_lora(const W16TileArgs& a, bool nv, bool out_bf16, hipStream_t stream);

}  // namespace mxf
