// What the product of two quantised matrices decides in whole numbers: which kernel a call of fp4_gemm launches (tile
// shape and K slices by its sizes), where its copies land and what a lane reads. Plain functions that also compile for
// the host (tests/test_fp4_pair_replay.py runs these very ones).
#pragma once

#include "w4a16_plan.hpp"

namespace mxf {

// bm == 32: the kernel of few tiles (32 x 32); slices > 1: sums of K slices through the workspace
struct Fp4PairPlan {
  int bm, bn, slices;
};

// What the launches are held to: fp4_gemm takes at most kMostTiles tiles of 128 x 128 (four times as many
// of 64 x 64, of 256 threads each: 2^31), and the kernel of 32 x 32 tiles never wins with more than a few rounds of the chip
constexpr int64_t kMostTiles = int64_t(1) << 21, kMostFewTiles = 4096;

// The shape with the least estimated time: a launch, then for each 256-k stage the length of one
// workgroup's stage (copy, barrier, decoding and MFMAs after each other) or, with k workgroups for each
// compute unit, their k shares of its work, whichever is longer; K slices add their sum's launch and
// traffic. Below the constants (us), fitted to these times (us: 32 x 32 | 64 x 64 | 64 x 128 | 128 x 128 |
// 256 x 256; 4s: 64 x 128 in 4 slices):
//                      NVFP4                               MXFP4
//   128 x 7168 x 4096    24 | 20 | 25 | 35 | 54              16 | 11 | 13 | 15 | 20
//   256 x 2048 x 2048    7.8 | 11 | 13 | 19 | 46             6.2 | 5.9 | 6.8 | 9.0 | 17
//   256 x 4096 x 7168    38 | 34 | 41 | 57 | 149  4s 31      23 | 17 | 20 | 23 | 45  4s 18
//   512 x 1024 x 16384   36 | 66 | 85 | 126 | 333  4s 33     24 | 34 | 40 | 49 | 95  4s 18
//   512 x 4096 x 7168    72 | 50 | 43 | 58 | 149             44 | 18 | 21 | 24 | 45
//   1024 x 2048 x 2048   28 | 16 | 15 | 20 | 46              21 | 7.4 | 7.4 | 9.7 | 17
//   1024 x 4096 x 7168   129 | 87 | 72 | 64 | 150            81 | 31 | 25 | 27 | 45
//   2000 x 4096 x 2048   98 | 53 | 45 | 36 | 50              75 | 20 | 17 | 14 | 18
//   3000 x 3008 x 4096   175 | 107 | 97 | 90 | 90            122 | 39 | 38 | 35 | 30
//   4096 x 4096 x 7168   489 | 329 | 280 | 225 | 199         312 | 116 | 94 | 78 | 65
inline Fp4PairPlan fp4_pair_plan(int64_t M, int64_t N, int64_t K, bool nv) {
  struct Shape {
    int bm, bn;
    float stage[2], work[2];  // MXFP4, NVFP4
  };
  constexpr Shape kShapes[] = {{32, 32, {0.14f, 0.27f}, {0.165f, 0.29f}},
                               {64, 64, {0.48f, 0.98f}, {0.245f, 0.68f}},
                               {64, 128, {0.58f, 1.35f}, {0.40f, 1.1f}},
                               {128, 128, {0.75f, 1.9f}, {0.65f, 1.88f}},
                               {256, 256, {1.6f, 5.2f}, {2.1f, 6.4f}}};
  const int64_t stages = w16_cdiv(K, 256);
  Fp4PairPlan best{256, 256, 1};
  float least = 3.0e38f;
  for (const Shape& t : kShapes) {
    const int64_t tiles = w16_cdiv(M, t.bm) * w16_cdiv(N, t.bn);
    if (t.bm == 32 && tiles > kMostFewTiles) continue;
    for (int s = 1; s <= 8 && s <= stages; s *= 2) {
      if (s > 1 && (t.bm == 32 || tiles * s > 512)) break;
      const float units = (float)(tiles * s) / 256.0f, k = units > 1.0f ? (float)w16_cdiv(tiles * s, 256) : units;
      const float stage = t.stage[nv] > k * t.work[nv] ? t.stage[nv] : k * t.work[nv];
      float us = 3.0f + (float)w16_cdiv(stages, s) * stage;
      if (s > 1) us += 4.5f + (float)s * (float)M * (float)N * 8.0f / 5.0e6f;
      if (us < least) {
        least = us;
        best = {t.bm, t.bn, s};
      }
    }
  }
  return best;
}

// ---- a stage of 256 k: 128 bytes of codes a row -------------------------------------------------------

// 16-byte copy number `chunk` of an operand's slot (row after row, 8 a row): where in the stage its bytes lie, the 8 of a
// row swapped among themselves
MXF_BOTH int64_t pair_copy_from(int chunk, int64_t wrow) {
  const int r = chunk >> 3;
  return r * wrow + 16 * ((chunk & 7) ^ swz_a16(r));
}

// Row r's 32-block 4 g + s of the stage, byte offset in the slot
MXF_BOTH int pair_block_at(int r, int g) { return r * 128 + 16 * ((4 * g) ^ swz_a16(r)); }
MXF_BOTH constexpr int pair_step(int at, int s) { return at ^ (16 * s); }

// lane group g's blocks of stage st lie past K (K ends in the middle of the last stage): its scales count as zero
MXF_BOTH bool pair_past(int g, int st, int64_t K) { return g == 1 && (int64_t)st * 256 + 128 >= K; }

// ---- scales: groups of 32 bytes a row, of 4 stages (MXFP4) or 2 (NVFP4) ---------------------------------

MXF_BOTH constexpr int pair_group_stages(bool nv) { return nv ? 2 : 4; }
MXF_BOTH constexpr int pair_scale_words(bool nv) { return nv ? 2 : 1; }  // dwords of a row, stage and lane group

// Part p of a group's copies (32 rows, 16 bytes a lane): where in the group a lane's bytes lie. 32 rows' first 16 bytes
// land beside each other, then their second: neighbouring rows on other banks
MXF_BOTH int64_t pair_scales_from(int p, int lane, int64_t srow) { return (32 * p + (lane & 31)) * srow + 16 * (lane >> 5); }

// The scales of row r, stage st and lane group g, byte offset in the group's slot: of row 0 and of the row in it
MXF_BOTH int pair_scales_at(int st, int g, bool nv) {
  const int off = 32 / pair_group_stages(nv) * (st % pair_group_stages(nv)) + 4 * pair_scale_words(nv) * g;
  return 512 * (off >> 4) + (off & 15);
}
MXF_BOTH constexpr int pair_scales_row(int r) { return 1024 * (r >> 5) + 16 * (r & 31); }

// the same in the kernel of few tiles, which loads them into registers: byte offset in the matrix
MXF_BOTH uint32_t pair_few_scales(int r, int g, int64_t srow, bool nv) { return (uint32_t)(r * srow) + 4 * pair_scale_words(nv) * g; }
MXF_BOTH uint32_t pair_few_scales_step(int st, bool nv) { return (uint32_t)st * 8 * pair_scale_words(nv); }
// its copies and loads of a stage, in this order: at most as many may be in flight when the stage before is read
constexpr int kFewCopies = 8, kFewLoads = 2;

// ---- results: 32 rows x `chunks` 16-byte pieces through LDS ------------------------------------------------

// fragment f's columns 8 j + 4 g .. + 3 of row r (bf16: 8 bytes, fp32: 16)
MXF_BOTH int pair_out_to(int f, int j, int g, int r, int es, int chunks) {
  const int c = es == 2 ? 4 * f + j : 8 * f + 2 * j + g;
  return 16 * chunks * r + 16 * (c ^ (r & (chunks - 1))) + (es == 2 ? 8 * g : 0);
}
// piece c of row r
MXF_BOTH int pair_out_from(int r, int c, int chunks) { return 16 * chunks * r + 16 * (c ^ (r & (chunks - 1))); }

// the kernel of few tiles: element (r, c) in a wave's sums, accumulator v of lane l at 65 v + l
MXF_BOTH int pair_few_sum(int r, int c) { return 65 * (4 * (c >> 3) + (c & 3)) + r + 32 * ((c >> 2) & 1); }

}  // namespace mxf
