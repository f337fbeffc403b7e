// Which kernel a call of fp4_gemm launches: tile shape and K slices by its sizes (host).
#pragma once

#include "common.hpp"

namespace mxf {

struct Fp4PairPlan {
  int bm, bn, slices;
};

inline Fp4PairPlan fp4_pair_plan(int64_t M, int64_t N, int64_t K, bool nv) {
  const int64_t t256 = cdiv(M, 256) * cdiv(N, 256), stages = cdiv(K, 256);
  if (t256 >= 192) return {256, 256, 1};
  const int64_t t128 = cdiv(M, 128) * cdiv(N, 128);
  int64_t s = t128 >= 256 ? 1 : 512 / t128;
  if (s > stages / 2) s = stages / 2;
  if (s > 16) s = 16;
  if (s < 1) s = 1;
  (void)nv;
  return {128, 128, (int)s};
}

}  // namespace mxf
