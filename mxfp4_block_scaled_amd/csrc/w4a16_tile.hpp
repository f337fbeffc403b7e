// Arguments and work lookup of the FP4-weight x bf16-activation kernels over ragged rows
// (w4a16_tile_body.hpp, w4a16_tile.hip, w4a16_grouped.hip, w4a16_lora.hip).
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
  const float* low;         // [lslices][R][rank]: scaling * a . lora_a^T, K slice by K slice
  int rank, L, S, lslices;
  int kslices;              // K slices of a sliced product
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

// Units of an expert of c rows in a launch for experts of lo_rows < c <= hi_rows
template <int BM>
__device__ __forceinline__ int w16_units(int c, int lo_rows, int hi_rows) {
  return c <= lo_rows || c > hi_rows ? 0 : (c + BM - 1) / BM;
}

// the first of n items that belongs to share i of s
__device__ __forceinline__ uint32_t w16_share(uint32_t n, int i, int s) { return n * (uint32_t)i / (uint32_t)s; }

// x n / 8 without leaving 32 bits
__device__ __forceinline__ uint32_t w16_eighths(uint32_t n, int x) {
  return (n >> 3) * (uint32_t)x + (((n & 7u) * (uint32_t)x) >> 3);
}

// Item w of units x ntiles items: groups of 8 units, n-tile by n-tile in a group, so that the some
// 64 items that an XCD has at work are about 8 units x 8 n-tiles, which take the fewest bytes
// into its L2. N-tile by n-tile over all units, an XCD reads all of the activations: 4096 x 4096 x
// 7168 with adapters 250 us, so 241; 8192 rows 433, 416; 8192 rows over 2 experts 436, 424; 16 units
// 244, 421, 426. Groups of n-tiles instead lose where an expert has few units (32 experts of 384
// rows 621, 635). ntiles x 8 stays in 32 bits: ntiles < 2^25.
__device__ __forceinline__ void w16_place(uint32_t w, uint32_t units, uint32_t ntiles, int& n_tile, int& unit) {
  constexpr uint32_t kGroup = 8;
  const uint32_t grp = w / (ntiles * kGroup), rem = w - grp * ntiles * kGroup;
  const uint32_t width = min(kGroup, units - grp * kGroup), n = rem / width;
  n_tile = (int)n;
  unit = (int)(grp * kGroup + rem - n * width);
}

// Item j of XCD x: the units' items (in an expert of more than 16 rows as w16_place puts them, else
// n-tile by n-tile) are split into 8 contiguous ranges, one per XCD, so that the workgroups of an
// XCD share activation rows and weight tiles in its L2. Called by whole waves; false: none.
// Every workgroup starts with this, so its latency counts: with CE > 0 (E <= 64 CE) each
// lane takes its experts' offsets in one batch of loads and keeps them.
template <int BM, int CE>
__device__ __forceinline__ bool w16_item_of(const int32_t* __restrict__ off, int E, int64_t R, int lo_rows, int hi_rows,
                                            int ntiles, int x, int j, int& e_out, int& n_out, int64_t& row0, int& m) {
  const int lane = threadIdx.x & 63;
  const int C = CE > 0 ? CE : (E + 63) >> 6, first = lane * C;
  int64_t r0 = 0;
  int units = 0;
  int o[CE + 1];  // CE > 0: the lane's row bounds (experts past E are empty)
  if constexpr (CE > 0) {
#pragma unroll
    for (int i = 0; i <= CE; ++i) o[i] = off[min(first + i, E)];
#pragma unroll
    for (int i = 0; i <= CE; ++i) {
      o[i] = min(max(o[i], 0), (int)R);
      if (i > 0) {
        o[i] = max(o[i], o[i - 1]);
        units += w16_units<BM>(o[i] - o[i - 1], lo_rows, hi_rows);
      }
    }
  } else {
    for (int i = 0; i < C; ++i)
      if (first + i < E) units += w16_units<BM>(w16_rows(off, R, first + i, r0), lo_rows, hi_rows);
  }
  int incl = units;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(incl, d);
    if (lane >= d) incl += y;
  }
  const int excl = incl - units;
  // the host keeps units x ntiles below 2^31; x total / 8 in 32 bits
  const uint32_t total = (uint32_t)__builtin_amdgcn_readlane(incl, 63) * (uint32_t)ntiles;
  const uint32_t w = w16_eighths(total, x) + (uint32_t)j;
  if (w >= w16_eighths(total, x + 1)) return false;
  const int p = (int)(w / (uint32_t)ntiles);
  const bool mine = p >= excl && p < incl;
  const unsigned long long msk = __ballot(mine);
  if (msk == 0) return false;
  const int src = __ffsll((long long)msk) - 1;
  int ee = 0, ue = 0, ke = 1, c = 0, lo = 0;
  if (mine) {
    int acc = excl;
#pragma unroll
    for (int i = 0; i < (CE > 0 ? CE : 1024); ++i) {
      if (CE == 0 && (i >= C || first + i >= E)) break;
      int ci;
      if constexpr (CE > 0) {
        r0 = o[i];
        ci = o[i + 1] - o[i];
      } else {
        ci = w16_rows(off, R, first + i, r0);
      }
      const int n = w16_units<BM>(ci, lo_rows, hi_rows);
      if (p >= acc && p < acc + n) {
        ee = first + i;
        ue = acc;
        ke = n;
        c = ci;
        lo = (int)r0;
      }
      acc += n;
    }
  }
  e_out = __builtin_amdgcn_readlane(ee, src);
  ue = __builtin_amdgcn_readlane(ue, src);
  ke = __builtin_amdgcn_readlane(ke, src);
  c = __builtin_amdgcn_readlane(c, src);
  lo = __builtin_amdgcn_readlane(lo, src);
  const uint32_t local = w - (uint32_t)ue * (uint32_t)ntiles;
  int loc;
  if constexpr (BM >= 64) {
    w16_place(local, (uint32_t)ke, (uint32_t)ntiles, n_out, loc);
  } else {
    n_out = (int)(local / (uint32_t)ke);
    loc = (int)(local - (uint32_t)n_out * (uint32_t)ke);
  }
  if (n_out < 0 || n_out >= ntiles || loc < 0) return false;
  row0 = lo + (int64_t)loc * BM;
  m = min(BM, c - loc * BM);
  return m > 0;
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
    const int step = (hi - lo + 63) / 64;
    const int64_t idx = lo + (int64_t)lane * step;
    const bool p = idx < hi && (int64_t)seg_off[idx < hi ? idx + 1 : 0] > t;
    const unsigned long long m = __ballot(p);
    const int probes = (hi - lo + step - 1) / step;
    const int f = m ? __ffsll((long long)m) - 1 : probes;  // the first probe past t
    const int nlo = f == 0 ? lo : lo + (f - 1) * step + 1;
    hi = f == probes ? hi : lo + f * step;
    lo = nlo;
    if (step == 1) break;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// tiles of rows x weight rows (64 x 128 without SwiGLU only)
enum class W16Shape { k64x128, k64x256, k128x256 };
void launch_w16_tile_grouped(const W16TileArgs& a, bool nv, bool swiglu, bool out_bf16, W16Shape shape, int64_t units,
                             hipStream_t stream);
void launch_w16_tile_lora(const W16TileArgs& a, bool nv, bool out_bf16, hipStream_t stream);

}  // namespace mxf
