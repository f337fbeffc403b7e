// What the FP4-weight x bf16-activation kernels over ragged rows decide in whole numbers: which
// kernels a call launches, which item a workgroup takes, where a copy lands and what it waits for.
// Plain functions that also compile for the host (tests/test_w4a16_plan.py runs these very ones).
#pragma once

#include <stdint.h>

#if defined(__HIP__)
#define MXF_BOTH __host__ __device__ __forceinline__
#else
#define MXF_BOTH inline
#endif

namespace mxf {

template <typename T>
MXF_BOTH T w16_min(T a, T b) { return a < b ? a : b; }
template <typename T>
MXF_BOTH T w16_max(T a, T b) { return a > b ? a : b; }
MXF_BOTH int64_t w16_cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ---- which kernels a call launches (host) ---------------------------------------------------------

// Threads of a launch: the runtime counts them in 32 bits
constexpr int64_t kMaxThreads = (int64_t(1) << 32) - 1;

// One launch over the experts of min_rows < rows <= max_rows: workgroups of bm rows x bn weight rows
// (bm == 16: the streaming kernel; else tiles, 64 x 128 without SwiGLU only)
struct W16Launch {
  int bm, bn, min_rows, max_rows;
  int64_t units, ntiles;
  int64_t workgroups() const { return 8 * w16_cdiv(units * ntiles, 8); }
  bool fits() const { return workgroups() * 256 <= kMaxThreads; }
};

// units of bm rows (0: whole experts) that experts of more than lo rows can make of R rows in all
inline int64_t w16_most_units(int64_t R, int E, int64_t lo, int bm) {
  const int64_t experts = R / (lo + 1) < E ? R / (lo + 1) : E;
  return bm == 0 ? experts : experts + R / bm;
}

// What the experts hold is on the device, so by bounds on it.
// Measured in us (8 experts: rows in all; streamed | 64 x 128 | 64 x 256 | 128 x 256 tiles):
//   2048 x 2048, 512 rows   18 | 20 | 24 | 33     4 experts 4096 x 7168, 512 rows   90 | 59 | 65 | 96
//                1024       28 | 23 | 25 | 34                            2048      351 | 144 | 155 | 154
//                6000      139 | 60 | 56 | 57                            6000      977 | 411 | 354 | 308
// The streaming kernel's time grows with workgroups x K (5 us a million) and needs one launch;
// a tiled launch lasts at least its K chain (0.36 us for 64 k of 64 x 128 tiles). Between them, where
// about half of the experts hold at most 16 rows, the streaming and the tiled launch follow each other
// with half of the weights each: 32 experts of 4096 x 4096, 256, 384, 512, 768 and 1024 rows 64, 84, 85,
// 83 and 79 us (NVFP4 80, 107, 109, 101, 100).
inline bool w16_streams_all(int64_t R, int64_t workgroups, int64_t K) {
  return R <= 128 || workgroups <= 1100 + 600000 / K;
}

// A short K (at most one super-step a wave) leaves a streaming workgroup little between its lookup and
// its sums: where there are many, each takes four runs of 64 MXFP4 weight rows. Measured in us, one
// and a half rows an expert, one | four runs:
//   workgroups    K 512          1024         1536         2048         2560         4096         7168
//    4096       28.2 | 34.7  36.7 | 42.7  42.2 | 48.9  53.2 | 66.3  66.7 | 83.8  91.3 | 116   157 | 188
//    8192       56.2 | 55.8  70.9 | 70.0  80.8 | 85.6   104 | 101    127 | 136    176 | 187   299 | 315
//   16384        108 | 102    137 | 128    155 | 156    195 | 187    240 | 248    340 | 347   585 | 613
//   28672        183 | 165    235 | 211    263 | 260    330 | 316    409 | 413    585 | 600  1045 | 1088
// NVFP4, whose decoding hides the lookup: 76.1 | 84.6, 93.3 | 102 and 126 | 136 at 8192 workgroups of K
// 512, 1024 and 2048, 245 | 239, 308 | 298 and 427 | 432 at 28672: always one.
inline int w16_stream_runs(int64_t units, int64_t N, int64_t K, bool nv) {
  return !nv && K <= 2048 && units * w16_cdiv(N, 64) >= 8192 ? 4 : 1;
}

// The launches of a grouped call, in order; returns how many
inline int w16_grouped_plan(int64_t R, int E, int64_t N, int64_t K, bool nv, bool swiglu, W16Launch (&l)[3]) {
  constexpr int kAll = 0x7FFFFFFF;
  const bool all = w16_streams_all(R, w16_most_units(R, E, 0, 16) * w16_cdiv(N, 64), K);
  const int64_t su = w16_most_units(R, E, 0, all ? 16 : 0);  // units of 16 rows read an expert's weights again from the cache
  const int runs = w16_stream_runs(su, N, K, nv);
  l[0] = W16Launch{16, 64 * runs, 0, all ? kAll : 16, su, w16_cdiv(N, 64 * runs)};
  if (all) return 1;
  const int64_t nt = w16_cdiv(N, 256), w128 = w16_most_units(R, E, 16, 128) * nt;
  if (w128 < 1024) {  // few tiles: one tiled launch, of the shape that keeps the chip busy
    int bm = 64, bn = 256;
    if (R >= 96 * (int64_t)E && w128 >= 384) bm = 128;
    else if (!swiglu && w16_most_units(R, E, 16, 64) * nt < 600) bn = 128;
    l[1] = W16Launch{bm, bn, 16, kAll, w16_most_units(R, E, 16, bm), w16_cdiv(N, bn)};
    return 2;
  }
  // A large call, perhaps a skewed one: by the expert's own rows. Measured in us against one 128 x 256
  // launch for all of more than 16 rows: top 6 of 256 experts of 7168 x 2048, 2048 tokens 556 | 581, Zipf
  // 446 | 448, 1024 tokens 501 | 526, Zipf 298 | 288; of 4096 x 7168 with SwiGLU, 2048 tokens 1099 | 1171,
  // Zipf 865 | 876, 4096 tokens 1571 | 1567, Zipf 1444 | 1423; of 64 of 4096 x 4096, 1024 tokens 238 |
  // 235, Zipf 288 | 272; of 32 of 4096 x 7168, 2048 tokens 615 | 612. NVFP4 alike.
  l[1] = W16Launch{64, 256, 16, 64, w16_most_units(R, E, 16, 0), nt};
  l[2] = W16Launch{128, 256, 64, kAll, w16_most_units(R, E, 64, 128), nt};
  return 3;
}

// Adapters: kernels, K slices and tiles of a call
struct W16LoraPlan {
  int base_slices;  // K slices of the projection's 64 x 128 tiles (0: whole tiles of bm x bn)
  int low_slices;   // K slices of the first product
  int low_rows;     // rows of a workgroup of the first product
  int low_share;    // workgroups that share a row block's segments
  int bm, bn;
  bool fits;        // every launch has fewer threads than the runtime counts
};

constexpr int kMaxBaseSlices = 8, kMaxLowSlices = 16, kMaxTileLowSlices = 4;

// Fewer than 256 tiles of 64 x 128, where the pass over the rows does not read lora_b too often
// (N x rank for each row, from the cache). Measured in us, sliced | whole tiles:
//   200 rows of 4096 x 7168, rank 16 and 64      30 | 63, 38 | 89     rank 128, 10 and 100 segments  56 | 127, 74 | 210
//   500 rows of 2048 x 2048, rank 16 and 64      25 | 27, 37 | 39     rank 128, 10 and 200 segments  58 | 58, 64 | 145
//   777 rows of 1520 x 2048, 101 segments, rank 24     31 | 39        rank 128  73 | 88
//   1000 rows of 1024 x 4096, rank 64, and rank 32 with 400 segments  45 | 47, 44 | 73     rank 128  66 | 63
//   3000 rows of 512 x 2048, rank 32                   34 | 28        rank 128  77 | 53
//   120 rows of 7168 x 2048, rank 64                   30 | 46        250 rows  49 | 47
// The left column is sliced by this rule, the right one is not; with a long K or many segments the
// border could lie higher.
inline bool w16_lora_sliced(int64_t M, int64_t N, int rank) {
  return M <= 64 || (w16_cdiv(M, 64) * w16_cdiv(N, 128) < 256 && M * N * rank <= (int64_t(1) << 26));
}

// Rows of a workgroup of the first product (not sliced): 32 where segments are long, so that an
// adapter is read for twice the rows, and where 16 (of 1024 threads) would be more threads than a launch has
inline bool w16_lora_wide(int64_t M, int64_t S) { return M >= 32 * S || M >= int64_t(1) << 26; }

inline int w16_clamp_slices(int64_t want, int64_t most) {
  return (int)(want < most ? (want > 1 ? want : 1) : (most > 1 ? most : 1));
}

// the most that a call of these sizes takes, whatever its S
inline int w16_lora_low_slices(int64_t M, int64_t N, int64_t K, int rank) {
  // sliced: K slices of at least 256 (64 for each of a workgroup's 4 waves), as many as fit the
  // compute units beside the projection's tiles. Else, with blocks of 32 rows, about a workgroup
  // a compute unit, each slice of at least 1024
  if (w16_lora_sliced(M, N, rank)) return w16_clamp_slices(512 / w16_cdiv(M, 16), w16_min<int64_t>(K / 256, kMaxLowSlices));
  return w16_clamp_slices(256 / w16_cdiv(M, 32), w16_min<int64_t>(K / 1024, kMaxTileLowSlices));
}

inline int w16_lora_base_slices(int64_t M, int64_t N, int64_t K, int rank) {
  // K slices of at least 256 for two workgroups a compute unit
  if (!w16_lora_sliced(M, N, rank)) return 0;
  return w16_clamp_slices(512 / (w16_cdiv(M, 64) * w16_cdiv(N, 128)), w16_min<int64_t>(K / 256, kMaxBaseSlices));
}

inline W16LoraPlan w16_lora_plan(int64_t M, int64_t N, int64_t K, int rank, int64_t S) {
  W16LoraPlan p{};
  p.base_slices = w16_lora_base_slices(M, N, K, rank);
  p.low_slices = w16_lora_low_slices(M, N, K, rank);
  if (p.base_slices > 0) {
    p.low_rows = 16;
    const int64_t blocks = w16_cdiv(M, 16);
    p.low_share = (int)w16_max<int64_t>(1, w16_min<int64_t>(16, w16_cdiv(S, blocks)));
    // what fits the compute units beside the projection's tiles
    p.low_slices = (int)w16_min<int64_t>(p.low_slices, w16_max<int64_t>(1, 512 / (blocks * p.low_share)));
    p.bm = 64;
    p.bn = 128;
    p.fits = true;  // M < 2^14
    return p;
  }
  const bool wide = w16_lora_wide(M, S);
  if (!wide) p.low_slices = 1;  // short segments: every slice is another pass over their adapters
  p.low_rows = wide ? 32 : 16;
  p.low_share = (int)w16_max<int64_t>(1, w16_min<int64_t>(16, w16_cdiv(S, w16_cdiv(M, p.low_rows))));
  // long segments: a block over the end of one has a second workgroup on the same compute unit
  // instead of twice the time (4096 x 4096 x 7168, 16 segments, 8 waves each: 250 -> 246 us)
  if (wide && S > 1 && p.low_share < 2) p.low_share = 2;
  // 128 x 256 tiles once there is about one for each of the 256 compute units (two fit one);
  // below that the small tile's four times as many workgroups finish sooner. Measured, us (64 x
  // 128 | 128 x 256): 4096 x 7168, 1500 rows 123 | 136, 2048 rows (256 tiles) 179 | 147, 8192 rows
  // 571 | 435; 2048 x 4096, 3000 rows (192 tiles) 75 | 83, 4096 rows 103 | 85. 256 x 256 tiles, one a
  // compute unit: 227 instead of 234 at 4096 x 4096 x 7168, where they fill the chip once, else slower.
  const bool large = w16_cdiv(M, 128) * w16_cdiv(N, 256) >= 240;
  p.bm = large ? 128 : 64;
  p.bn = large ? 256 : 128;
  p.fits = 8 * w16_cdiv(w16_cdiv(M, p.low_rows), 8) * (wide ? 512 : 1024) <= kMaxThreads &&
           W16Launch{p.bm, p.bn, 0, 0, w16_cdiv(M, p.bm), w16_cdiv(N, p.bn)}.fits();
  return p;
}

// ---- which item a workgroup takes ------------------------------------------------------------------

// Rows of expert e as stored, held inside [0, R): offsets that are not ascending or leave
// the range cannot lead outside the operands.
MXF_BOTH int w16_rows(const int32_t* __restrict__ off, int64_t R, int e, int64_t& lo) {
  lo = w16_min(w16_max((int64_t)off[e], (int64_t)0), R);
  const int64_t hi = w16_min(w16_max((int64_t)off[e + 1], lo), R);
  return (int)(hi - lo);
}

// Units of an expert of c rows in a launch for experts of lo_rows < c <= hi_rows
template <int BM>
MXF_BOTH int w16_units(int c, int lo_rows, int hi_rows) {
  return c <= lo_rows || c > hi_rows ? 0 : (int)(((int64_t)c + BM - 1) / BM);
}

// the first of n items that belongs to share i of s
MXF_BOTH uint32_t w16_share(uint32_t n, int i, int s) { return n * (uint32_t)i / (uint32_t)s; }

// x n / 8 without leaving 32 bits
MXF_BOTH uint32_t w16_eighths(uint32_t n, int x) {
  return (n >> 3) * (uint32_t)x + (((n & 7u) * (uint32_t)x) >> 3);
}

// Item w of units x ntiles items: groups of 8 units, n-tile by n-tile in a group, so that the about
// 64 items that an XCD has at work are 8 units x 8 n-tiles, which take the fewest bytes into its L2.
// 4096 x 4096 x 7168 with adapters 241 us; 250 with the n-tiles of all units after each other, where
// an XCD reads all of the activations. 8192 rows 416 and 433; 8192 rows over 2 experts 424 and 436.
// Groups of 16 units: 244, 421, 426. Groups of n-tiles instead lose where an expert has few units (32
// experts of 384 rows 621, 635). ntiles x 8 stays in 32 bits: ntiles < 2^25.
MXF_BOTH void w16_place(uint32_t w, uint32_t units, uint32_t ntiles, int& n_tile, int& unit) {
  constexpr uint32_t kGroup = 8;
  const uint32_t grp = w / (ntiles * kGroup), rem = w - grp * ntiles * kGroup;
  const uint32_t width = w16_min(kGroup, units - grp * kGroup), n = rem / width;
  n_tile = (int)n;
  unit = (int)(grp * kGroup + rem - n * width);
}

// Item j of XCD x of `total` items (8 contiguous ranges, one per XCD); false: none
MXF_BOTH bool w16_range(uint32_t total, int x, int j, uint32_t& w) {
  w = w16_eighths(total, x) + (uint32_t)j;
  return w < w16_eighths(total, x + 1);
}

// The lookup's share of one lane of a wave: experts lane C .. lane C + C - 1. With CE > 0 (E <= 64 CE)
// it takes their row bounds in one batch of loads and keeps them (o; experts past E are empty).
template <int CE>
MXF_BOTH int w16_lane_experts(int E) {
  return CE > 0 ? CE : (E + 63) >> 6;
}

template <int BM, int CE>
MXF_BOTH int w16_lane_units(const int32_t* __restrict__ off, int E, int64_t R, int lo_rows, int hi_rows, int lane,
                            int (&o)[CE + 1]) {
  const int C = w16_lane_experts<CE>(E), first = lane * C;
  int units = 0;
  if constexpr (CE > 0) {
#pragma unroll
    for (int i = 0; i <= CE; ++i) o[i] = off[w16_min(first + i, E)];
#pragma unroll
    for (int i = 0; i <= CE; ++i) {
      o[i] = w16_min(w16_max(o[i], 0), (int)R);
      if (i > 0) {
        o[i] = w16_max(o[i], o[i - 1]);
        units += w16_units<BM>(o[i] - o[i - 1], lo_rows, hi_rows);
      }
    }
  } else {
    int64_t r0;
    for (int i = 0; i < C; ++i)
      if (first + i < E) units += w16_units<BM>(w16_rows(off, R, first + i, r0), lo_rows, hi_rows);
  }
  return units;
}

// The expert that holds unit p, which is one of the lane's: units before it, its units, rows and first row
struct W16Pick {
  int e, before, units, rows, row0;
};

template <int BM, int CE>
MXF_BOTH W16Pick w16_lane_find(const int32_t* __restrict__ off, int E, int64_t R, int lo_rows, int hi_rows, int lane,
                               const int (&o)[CE + 1], int before, int p) {
  const int C = w16_lane_experts<CE>(E), first = lane * C;
  W16Pick k{0, 0, 1, 0, 0};
#pragma unroll
  for (int i = 0; i < (CE > 0 ? CE : 1024); ++i) {
    if (CE == 0 && (i >= C || first + i >= E)) break;
    int c;
    int64_t r0;
    if constexpr (CE > 0) {
      r0 = o[i];
      c = o[i + 1] - o[i];
    } else {
      c = w16_rows(off, R, first + i, r0);
    }
    const int n = w16_units<BM>(c, lo_rows, hi_rows);
    if (p >= before && p < before + n) k = W16Pick{first + i, before, n, c, (int)r0};
    before += n;
  }
  return k;
}

// n-tile and rows of item w in its expert (of more than 16 rows as w16_place puts them, else n-tile by
// n-tile); false: none (offsets that are not ascending)
template <int BM>
MXF_BOTH bool w16_item_place(const W16Pick& k, uint32_t w, int ntiles, int& n_tile, int64_t& row0, int& m) {
  const uint32_t local = w - (uint32_t)k.before * (uint32_t)ntiles;
  int unit;
  if constexpr (BM >= 64) {
    w16_place(local, (uint32_t)k.units, (uint32_t)ntiles, n_tile, unit);
  } else {
    n_tile = (int)(local / (uint32_t)k.units);
    unit = (int)(local - (uint32_t)n_tile * (uint32_t)k.units);
  }
  if (n_tile < 0 || n_tile >= ntiles || unit < 0) return false;
  row0 = k.row0 + (int64_t)unit * BM;
  m = (int)w16_min((int64_t)BM, (int64_t)k.rows - (int64_t)unit * BM);
  return m > 0;
}

// One step of the search for the first segment whose end lies past row t: lane i probes segment
// lo + i step, and the lanes' answers, a mask, narrow [lo, hi]
MXF_BOTH int w16_probe_step(int lo, int hi) { return (hi - lo + 63) / 64; }
MXF_BOTH bool w16_probe(const int32_t* __restrict__ seg_off, int lo, int hi, int lane, int64_t t) {
  const int64_t i = lo + (int64_t)lane * w16_probe_step(lo, hi);
  return i < hi && (int64_t)seg_off[i < hi ? i + 1 : 0] > t;
}
MXF_BOTH void w16_probe_narrow(unsigned long long mask, int& lo, int& hi) {
  const int step = w16_probe_step(lo, hi), probes = (hi - lo + step - 1) / step;
  const int f = mask ? __builtin_ctzll(mask) : probes;  // the first probe past t
  const int nlo = f == 0 ? lo : lo + (f - 1) * step + 1;
  hi = f == probes ? hi : lo + f * step;
  lo = nlo;
}

// ---- a tile's copies and waits ----------------------------------------------------------------------

MXF_BOTH constexpr int swz_a16(int r) { return (r & 7) ^ ((r >> 3) & 1); }  // 8 chunks per row
MXF_BOTH constexpr int swz_b16(int r) { return (r >> 2) & 3; }              // 4 chunks per row

// the weight row that row r of n-tile n holds (N and beyond: reads as zero); with SwiGLU gate rows, then up rows
MXF_BOTH int64_t w16_weight_row(bool swiglu, int BN, int64_t half, int n, int r) {
  if (swiglu) return (r < BN / 2 ? 0 : half - BN / 2) + (int64_t)n * (BN / 2) + r;
  return (int64_t)n * BN + r;
}

// Issue order at stage st, the i-th of whole turns of the slots (NA of activations, two of 128 k of
// codes and of a scale group of P stages): on even i the codes of stages st + 2, st + 3 and, where a
// scale group begins (or the slice does), the next group, then the activations of st + NA - 1.
MXF_BOTH constexpr bool w16_issues_codes(int i, int st, int nst) { return i % 2 == 0 && st + 2 < nst; }
MXF_BOTH constexpr bool w16_begins_scales(int st, int st0, int P, int nst) {
  return (st % P == 0 || st == st0) && (st / P + 1) * P < nst;
}
MXF_BOTH constexpr bool w16_issues_a(int st, int NA, int nst) { return st + NA - 1 < nst; }
MXF_BOTH constexpr int w16_a_slot(int i, int NA) { return i % NA; }
MXF_BOTH constexpr int w16_code_slot(int i) { return (i / 2) % 2; }
MXF_BOTH constexpr int w16_turn(int NA) { return NA == 3 ? 12 : 4; }
// Copies of a wave that may be in flight when stage st begins: with three slots those of the stage
// before, IA of activations and after an even stage IB of codes (and the scales) before them
MXF_BOTH constexpr int w16_in_flight(int i, int NA, int IA, int IB, bool last, bool scales) {
  return NA == 2 || last ? 0 : i % 2 == 0 ? IA : IA + IB + (scales ? 1 : 0);
}

}  // namespace mxf
