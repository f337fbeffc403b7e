// Sums and maxima over the 64 lanes of a wave on the VALU: four DPP steps inside each row of 16
// lanes, then gfx950's row and half swaps. Given x twice, a swap returns a pair whose two values
// are x of the lane and of its partner (in either order), so that combining the pair is the
// butterfly's step. Every lane ends with the same value, by the same tree.
#pragma once

#include "common.hpp"

namespace mxf {

template <int kCtrl>
__device__ __forceinline__ float dpp_move(float x) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), kCtrl, 0xF, 0xF, true));
#else
  return x;
#endif
}

template <typename Op>
__device__ __forceinline__ float wave_reduce(float x, Op op) {
  x = op(x, dpp_move<0xB1>(x));   // lanes 1 0 3 2 of each four
  x = op(x, dpp_move<0x4E>(x));   // lanes 2 3 0 1
  x = op(x, dpp_move<0x141>(x));  // eight lanes mirrored
  x = op(x, dpp_move<0x140>(x));  // sixteen lanes mirrored
#if defined(__HIP_DEVICE_COMPILE__)
  const uint32_t u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  x = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
  const uint32_t w = __float_as_uint(x);
  const auto h = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  x = op(__uint_as_float(h[0]), __uint_as_float(h[1]));
#endif
  return x;
}

__device__ __forceinline__ float wave_sum(float x) {
  return wave_reduce(x, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float wave_max(float x) {
  return wave_reduce(x, [](float a, float b) { return fmaxf(a, b); });
}

}  // namespace mxf
