// Which kernel a call of fp4_gemm launches: tile shape and K slices by its sizes (host).
#pragma once

#include "common.hpp"

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
  const int64_t stages = cdiv(K, 256);
  Fp4PairPlan best{256, 256, 1};
  float least = 3.0e38f;
  for (const Shape& t : kShapes) {
    const int64_t tiles = cdiv(M, t.bm) * cdiv(N, t.bn);
    if (t.bm == 32 && tiles > kMostFewTiles) continue;
    for (int s = 1; s <= 8 && s <= stages; s *= 2) {
      if (s > 1 && (t.bm == 32 || tiles * s > 512)) break;
      const float units = (float)(tiles * s) / 256.0f, k = units > 1.0f ? (float)cdiv(tiles * s, 256) : units;
      const float stage = t.stage[nv] > k * t.work[nv] ? t.stage[nv] : k * t.work[nv];
      float us = 3.0f + (float)cdiv(stages, s) * stage;
      if (s > 1) us += 4.5f + (float)s * (float)M * (float)N * 8.0f / 5.0e6f;
      if (us < least) {
        least = us;
        best = {t.bm, t.bn, s};
      }
    }
  }
  return best;
}

}  // namespace mxf
