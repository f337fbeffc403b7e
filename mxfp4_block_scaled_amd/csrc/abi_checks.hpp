// Argument checks shared by the extern "C" entry points.
#pragma once

#include "mxfp4_moe.h"

#include <hip/hip_runtime.h>

namespace mxf_abi {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline hipStream_t as_stream(mxf_stream s) { return reinterpret_cast<hipStream_t>(s); }

inline bool valid_elem(int f) { return f == MXF_E4M3 || f == MXF_E2M1; }
inline bool valid_weight(int f) { return f == MXF_W_MXFP4 || f == MXF_W_NVFP4; }
inline bool valid_dtype(int d) { return d == MXF_F32 || d == MXF_BF16; }

inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxOffset = int64_t(1) << 32;  // byte offsets that kernels keep in 32 bits stay below

template <int N>
inline bool all_aligned16(const void* const (&ptrs)[N]) {
  for (const void* p : ptrs)
    if (!aligned16(p)) return false;
  return true;
}

}  // namespace mxf_abi
