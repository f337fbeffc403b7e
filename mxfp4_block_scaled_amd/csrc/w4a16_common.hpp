// FP4 weights as bf16 matrix operands: the register decoders shared by the kernels that
// multiply FP4 weights with bf16 activations (gemm_w4a16.hip, w4a16_tile_body.hpp,
// w4a16_grouped.hip).
#pragma once

#include "gemm_common.hpp"

namespace mxf {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

// UE4M3 (OCP E4M3 with the sign bit clear) -> fp32, exact: exponent 0 is subnormal
// (m x 2^-9), otherwise 2^(e-7) (1 + m/8)
__device__ __forceinline__ float ue4m3_to_f32(uint32_t b) {
  const uint32_t e = (b >> 3) & 15u, m = b & 7u;
  const float sub = (float)m * 0.001953125f;
  const float nrm = __uint_as_float(((e + 120u) << 23) | (m << 20));
  return e == 0 ? sub : nrm;
}

// 2^(b - 127) as fp32 (b = 0: the subnormal 2^-127)
__device__ __forceinline__ float ue8m0_to_f32(uint32_t b) { return __uint_as_float(b ? b << 23 : 0x00400000u); }

typedef float v2f __attribute__((ext_vector_type(2)));

// 8 E2M1 codes (one dword, element 2n in the low nibble of byte n) x a power-of-two
// scale -> 8 bf16 (the scaled conversion applies only the exponent of its fp32 scale)
__device__ __forceinline__ v8bf decode8(uint32_t codes, float scale) {
#if defined(__HIP_DEVICE_COMPILE__)
  const v2bf p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
  const v2bf p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
  const v2bf p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
  const v2bf p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  return v8bf{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
#else
  (void)codes;
  (void)scale;
  return v8bf{};
#endif
}

// 8 E2M1 codes x a UE4M3 scale -> 8 bf16: the scale's power of two goes into the scaled
// conversion to fp32, its mantissa factor f = 1 + m/8 is multiplied in fp32 (both exact:
// a code times f has at most 5 significant bits), then each pair rounds to bf16 exactly
__device__ __forceinline__ v8bf decode8_nv(uint32_t codes, float scale) {
#if defined(__HIP_DEVICE_COMPILE__)
  const uint32_t sb = __float_as_uint(scale);
  const float p = __uint_as_float(sb & 0x7F800000u);               // 2^floor(log2 scale); 0 for 0
  const float f = __uint_as_float((sb & 0x007FFFFFu) | 0x3F800000u);  // scale / p in [1, 2)
  const v2f x0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, p, 0);
  const v2f x1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, p, 1);
  const v2f x2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, p, 2);
  const v2f x3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, p, 3);
  return v8bf{(__bf16)(x0[0] * f), (__bf16)(x0[1] * f), (__bf16)(x1[0] * f), (__bf16)(x1[1] * f),
              (__bf16)(x2[0] * f), (__bf16)(x2[1] * f), (__bf16)(x3[0] * f), (__bf16)(x3[1] * f)};
#else
  (void)codes;
  (void)scale;
  return v8bf{};
#endif
}

}  // namespace mxf
