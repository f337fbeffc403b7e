// Quantisation of a matrix to 4-bit block formats and back.
//
// NVFP4: blocks of 16 with a UE4M3 scale s = E4M3(amax / (6 g)), g the tensor's scale (fp32);
// MXFP4: blocks of 32 with a UE8M0 scale 2^(floor(log2 amax) - 2), g = 1. An element's code is the
// E2M1 value nearest to x / d, d = s g (ties to even), or with random bytes r the upper of its two
// neighbours where the part above the lower one exceeds (r + 1/2) / 256. Blocks lie along the rows,
// along the columns (the codes of x^T, rows filled up to 128), or both from one read of x.
//
// x / d is the correctly rounded quotient: q = x (1/d) and one Newton step with the exact remainder,
// q + (x - q d) (1/d). With the reciprocal alone a value halfway between two codes (often: x has 8
// bits and s 4) could land on either side of the tie.
//
// HBM-bound: x once, the codes and scales once. Where columns are wanted a workgroup holds a
// 128 x 128 tile of x in LDS; the codes along columns go back through LDS so that they leave as whole
// 64-byte pieces of a row of x^T.
#include "mx_codec.hpp"
#include "wave.hpp"
#include "w4a16_common.hpp"

namespace mxf {

namespace {

typedef unsigned int u4v __attribute__((ext_vector_type(4)));

constexpr float kTiny = 1.17549435e-38f;  // 2^-126

// what a block's elements are divided by
struct Divisor {
  float d, inv;
  uint32_t byte;
};

template <bool kNV>
__device__ __forceinline__ Divisor divisor_of(uint32_t amax_bits, float g) {
  Divisor v;
  if (kNV) {
    v.byte = e4m3_mag_code(__uint_as_float(amax_bits) / (6.0f * g));
    v.d = ue4m3_to_f32(v.byte) * g;
    if (!(v.d >= kTiny && v.d <= 3.0e38f)) {  // the block is stored as zeros (NaN and infinite g too)
      v.byte = 0;
      v.d = 0.0f;
      v.inv = 0.0f;
    } else {
      v.inv = 1.0f / v.d;
    }
  } else {
    v.byte = scale_byte_from_amax_bits(amax_bits, kEmaxE2M1);
    v.d = ue8m0_to_f32(v.byte);
    v.inv = inv_scale_from_byte(min(v.byte, 253u));
  }
  return v;
}

template <bool kNV>
__device__ __forceinline__ float quotient(float x, const Divisor& v) {
  const float q = x * v.inv;
  if (!kNV) return q;  // by a power of two: exact
  return copysignf(fmaf(fmaf(-q, v.d, x), v.inv, q), x);  // -0 loses its sign in the sum
}

// the stochastic choice between the two E2M1 neighbours of q, as a value
__device__ __forceinline__ float dither(float q, uint32_t r) {
  const float a = fabsf(q);
  const float step = a < 2.0f ? 0.5f : a < 4.0f ? 1.0f : 2.0f, per = a < 2.0f ? 2.0f : a < 4.0f ? 1.0f : 0.5f;
  const float u = a * per, low = floorf(u);
  const float n = low + ((u - low) * 256.0f > (float)r + 0.5f ? 1.0f : 0.0f);
  return copysignf(fminf(n * step, 6.0f), q);
}

// 8 values -> one dword of codes
__device__ __forceinline__ uint32_t pack8(const float (&x)[8]) {
  uint32_t w = 0;
#if defined(__HIP_DEVICE_COMPILE__)
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], 1.0f, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], 1.0f, 3);
#endif
  return w;
}

// One block of B values (and random bytes, four a word) -> B / 8 dwords of codes; returns the scale byte
template <bool kNV, bool kSR, int B>
__device__ __forceinline__ uint32_t quantise_block(const float (&x)[B], const uint32_t (&r)[B / 4], float g,
                                                   uint32_t (&out)[B / 8]) {
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < B; ++i) amax = max(amax, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  const Divisor v = divisor_of<kNV>(amax, g);
#pragma unroll
  for (int k = 0; k < B / 8; ++k) {
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = 8 * k + i;
      q[i] = quotient<kNV>(x[at], v);
      if (kSR) q[i] = dither(q[i], (r[at / 4] >> (8 * (at % 4))) & 0xFFu);
    }
    out[k] = pack8(q);
  }
  return v.byte;
}

template <bool kBF16, int N>
__device__ __forceinline__ void load_values(const void* p, int64_t at, float (&x)[N]) {
  const u4v* src = reinterpret_cast<const u4v*>(static_cast<const char*>(p) + at * (kBF16 ? 2 : 4));
#pragma unroll
  for (int i = 0; i < N / (kBF16 ? 8 : 4); ++i) {
    const u4v w = __builtin_nontemporal_load(src + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (kBF16) {
        x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
        x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      } else {
        x[4 * i + j] = __uint_as_float(w[j]);
      }
    }
  }
}

// Along rows only: one thread per block.
template <bool kBF16, bool kNV, bool kSR>
__global__ void __launch_bounds__(256) quantise_rows_kernel(Fp4QuantArgs a) {
  constexpr int B = kNV ? 16 : 32;
  const int64_t b = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (b >= a.rows * (a.cols / B)) return;
  const float g = a.tensor_scale ? *a.tensor_scale : 1.0f;
  float x[B];
  load_values<kBF16>(a.x, b * B, x);
  uint32_t r[B / 4] = {}, out[B / 8];
  if (kSR) {
#pragma unroll
    for (int i = 0; i < B / 16; ++i) {
      const u4v w = __builtin_nontemporal_load(reinterpret_cast<const u4v*>(a.rnd + b * B) + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) r[4 * i + j] = w[j];
    }
  }
  a.q_scale[b] = (uint8_t)quantise_block<kNV, kSR>(x, r, g, out);
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.q + b * (B / 2));
  if (kNV) *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
  else *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[B / 8 - 2], out[B / 8 - 1]);
}

// Along columns, and along rows where wanted: a 128 x 128 tile per workgroup.
template <bool kBF16, bool kNV, bool kSR>
__global__ void __launch_bounds__(256) quantise_both_kernel(Fp4QuantArgs a) {
  constexpr int B = kNV ? 16 : 32, T = 128, ES = kBF16 ? 2 : 4, RS = T * ES + 16;  // bytes of a row of the tile
  __shared__ __align__(16) uint8_t tile[T * RS];
  __shared__ __align__(16) uint8_t dice[kSR ? T * T : 16];
  __shared__ __align__(16) uint32_t codes[T][T / 8 + 1];
  __shared__ uint8_t scales[T][T / B];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t ct = (a.cols + T - 1) / T, row0 = (int64_t)(blockIdx.x / ct) * T, col0 = (int64_t)(blockIdx.x % ct) * T;
  const float g = a.tensor_scale ? *a.tensor_scale : 1.0f;

  // rows: a thread's block of B columns, 8 (4) threads a row
  constexpr int PR = T / B, RP = 256 / PR;
#pragma unroll 2
  for (int i = 0; i < T / RP; ++i) {
    const int r = RP * i + tid / PR, c = (tid % PR) * B;
    const int64_t row = row0 + r, col = col0 + c;
    const bool in = row < a.rows && col < a.cols;
    float x[B] = {};
    uint32_t dw[B / 4] = {};
    if (in) {
      load_values<kBF16>(a.x, row * a.cols + col, x);
      if (kSR) {
#pragma unroll
        for (int k = 0; k < B / 16; ++k) {
          const u4v w = __builtin_nontemporal_load(reinterpret_cast<const u4v*>(a.rnd + row * a.cols + col) + k);
#pragma unroll
          for (int j = 0; j < 4; ++j) dw[4 * k + j] = w[j];
        }
      }
    }
    uint8_t* at = tile + r * RS + c * ES;
    if (kBF16) {
#pragma unroll
      for (int k = 0; k < B / 8; ++k)
        *reinterpret_cast<u4v*>(at + 16 * k) =
            u4v{__float_as_uint(x[8 * k]) >> 16 | __float_as_uint(x[8 * k + 1]),
                __float_as_uint(x[8 * k + 2]) >> 16 | __float_as_uint(x[8 * k + 3]),
                __float_as_uint(x[8 * k + 4]) >> 16 | __float_as_uint(x[8 * k + 5]),
                __float_as_uint(x[8 * k + 6]) >> 16 | __float_as_uint(x[8 * k + 7])};
    } else {
#pragma unroll
      for (int k = 0; k < B / 4; ++k)
        *reinterpret_cast<u4v*>(at + 16 * k) = u4v{__float_as_uint(x[4 * k]), __float_as_uint(x[4 * k + 1]),
                                                   __float_as_uint(x[4 * k + 2]), __float_as_uint(x[4 * k + 3])};
    }
    if (kSR) {
#pragma unroll
      for (int k = 0; k < B / 16; ++k)
        *reinterpret_cast<u4v*>(dice + r * T + c + 16 * k) = u4v{dw[4 * k], dw[4 * k + 1], dw[4 * k + 2], dw[4 * k + 3]};
    }
    if (a.q && in) {
      uint32_t out[B / 8];
      const uint32_t byte = quantise_block<kNV, kSR>(x, dw, g, out);
      const int64_t b = (row * a.cols + col) / B;
      a.q_scale[b] = (uint8_t)byte;
      uint32_t* dst = reinterpret_cast<uint32_t*>(a.q + b * (B / 2));
      if (kNV) *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
      else *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[B / 8 - 2], out[B / 8 - 1]);
    }
  }
  __syncthreads();

  // columns: a lane's two columns, B rows at a time
#pragma unroll 1
  for (int i = wave; i < T / B; i += 4) {
    float x[2][B];
    uint32_t dw[2][B / 4] = {};
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const uint8_t* at = tile + (B * i + k) * RS + 2 * lane * ES;
      if (kBF16) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(at);
        x[0][k] = __uint_as_float(w << 16);
        x[1][k] = __uint_as_float(w & 0xFFFF0000u);
      } else {
        const uint2 w = *reinterpret_cast<const uint2*>(at);
        x[0][k] = __uint_as_float(w.x);
        x[1][k] = __uint_as_float(w.y);
      }
      if (kSR) {
        const uint32_t w = *reinterpret_cast<const uint16_t*>(dice + (B * i + k) * T + 2 * lane);
        dw[0][k / 4] |= (w & 0xFFu) << (8 * (k % 4));
        dw[1][k / 4] |= (w >> 8) << (8 * (k % 4));
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t out[B / 8];
      scales[2 * lane + h][i] = (uint8_t)quantise_block<kNV, kSR>(x[h], dw[h], g, out);
#pragma unroll
      for (int k = 0; k < B / 8; ++k) codes[2 * lane + h][B / 8 * i + k] = out[k];
    }
  }
  __syncthreads();

  // out: 64 bytes of codes and T / B scales of each column
  const int64_t padded = (a.rows + 127) / 128 * 128;
#pragma unroll
  for (int i = 0; i < T * 4 / 256; ++i) {
    const int idx = tid + 256 * i, c = idx >> 2, p = idx & 3;
    if (col0 + c < a.cols)
      *reinterpret_cast<uint4*>(a.qt + (col0 + c) * (padded / 2) + row0 / 2 + 16 * p) =
          make_uint4(codes[c][4 * p], codes[c][4 * p + 1], codes[c][4 * p + 2], codes[c][4 * p + 3]);
  }
  for (int idx = tid; idx < T * (T / B); idx += 256) {
    const int c = idx / (T / B), p = idx % (T / B);
    if (col0 + c < a.cols) a.qt_scale[(col0 + c) * (padded / B) + row0 / B + p] = scales[c][p];
  }
}

// 32 codes a thread -> values x block scale x tensor scale
template <bool kBF16, bool kNV>
__global__ void __launch_bounds__(256) dequantise_kernel(const uint8_t* q, const uint8_t* q_scale, int64_t n,
                                                         const float* tensor_scale, void* out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const float g = tensor_scale ? *tensor_scale : 1.0f;
  const u4v w = __builtin_nontemporal_load(reinterpret_cast<const u4v*>(q) + i);
  float s[2];
  if (kNV) {
    const uint32_t b = reinterpret_cast<const uint16_t*>(q_scale)[i];
    s[0] = ue4m3_to_f32(b & 0x7Fu);
    s[1] = ue4m3_to_f32((b >> 8) & 0x7Fu);
  } else {
    s[0] = s[1] = ue8m0_to_f32(q_scale[i]);
  }
  float v[32];
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const v2f p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[k], 1.0f, 0);
    const v2f p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[k], 1.0f, 1);
    const v2f p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[k], 1.0f, 2);
    const v2f p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[k], 1.0f, 3);
    const float e[8] = {p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
#pragma unroll
    for (int j = 0; j < 8; ++j) v[8 * k + j] = e[j] * s[k / 2] * g;
  }
#endif
  if (kBF16) {
    u4v* dst = reinterpret_cast<u4v*>(static_cast<uint16_t*>(out) + i * 32);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      __builtin_nontemporal_store(u4v{bf16x2_bits(v[8 * k], v[8 * k + 1]), bf16x2_bits(v[8 * k + 2], v[8 * k + 3]),
                                      bf16x2_bits(v[8 * k + 4], v[8 * k + 5]), bf16x2_bits(v[8 * k + 6], v[8 * k + 7])}, dst + k);
  } else {
    u4v* dst = reinterpret_cast<u4v*>(static_cast<float*>(out) + i * 32);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      __builtin_nontemporal_store(u4v{__float_as_uint(v[4 * k]), __float_as_uint(v[4 * k + 1]),
                                      __float_as_uint(v[4 * k + 2]), __float_as_uint(v[4 * k + 3])}, dst + k);
  }
}

// The largest magnitude, as bits: the maximum of integers is the same in any order.
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
  __shared__ uint32_t red[16];
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  m = 0;
  for (int w = 0; w < (int)(blockDim.x >> 6); ++w) m = max(m, red[w]);
  return m;
}

// the smallest power of two, 2^-126 at least, that takes amax to at most 6 x 448 = 21/16 x 2^11; 1 for 0
__device__ __forceinline__ float scale_of_amax(uint32_t amax) {
  if (amax == 0) return 1.0f;
  const int e = (int)(amax >> 23) - 11 + ((amax & 0x7FFFFFu) > 0x280000u ? 1 : 0);
  return __uint_as_float((uint32_t)max(e, 1) << 23);
}

template <bool kBF16>
__global__ void __launch_bounds__(512) amax_kernel(const u4v* x, int64_t n, uint32_t* partial, float* scale) {
  uint32_t m = 0;
  const int64_t step = (int64_t)gridDim.x * 512;
  for (int64_t i = (int64_t)blockIdx.x * 512 + threadIdx.x; i < n; i += 4 * step) {
    u4v w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = i + k * step < n ? x[i + k * step] : u4v{0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (kBF16) m = max(m, max((w[k][j] << 16) & 0x7FFFFFFFu, w[k][j] & 0x7FFF0000u));
        else m = max(m, w[k][j] & 0x7FFFFFFFu);
      }
  }
  m = block_max(m);
  if (threadIdx.x == 0) {
    if (gridDim.x == 1) *scale = scale_of_amax(m);
    else partial[blockIdx.x] = m;
  }
}

__global__ void __launch_bounds__(512) amax_finish_kernel(const uint32_t* partial, int n, float* scale) {
  uint32_t m = 0;
  for (int i = threadIdx.x; i < n; i += 512) m = max(m, partial[i]);
  m = block_max(m);
  if (threadIdx.x == 0) *scale = scale_of_amax(m);
}

template <bool kBF16, bool kNV, bool kSR>
void launch_quant_t(const Fp4QuantArgs& a, hipStream_t stream) {
  if (a.qt)
    quantise_both_kernel<kBF16, kNV, kSR><<<(unsigned)(cdiv(a.rows, 128) * cdiv(a.cols, 128)), 256, 0, stream>>>(a);
  else
    quantise_rows_kernel<kBF16, kNV, kSR><<<(unsigned)cdiv(a.rows * (a.cols / (kNV ? 16 : 32)), 256), 256, 0, stream>>>(a);
}

}  // namespace

int launch_fp4_quantize(const Fp4QuantArgs& a, bool x_bf16, bool nvfp4, hipStream_t stream) {
  const bool sr = a.rnd != nullptr;
  if (x_bf16) {
    if (nvfp4) sr ? launch_quant_t<true, true, true>(a, stream) : launch_quant_t<true, true, false>(a, stream);
    else sr ? launch_quant_t<true, false, true>(a, stream) : launch_quant_t<true, false, false>(a, stream);
  } else {
    if (nvfp4) sr ? launch_quant_t<false, true, true>(a, stream) : launch_quant_t<false, true, false>(a, stream);
    else sr ? launch_quant_t<false, false, true>(a, stream) : launch_quant_t<false, false, false>(a, stream);
  }
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_fp4_dequantize(const uint8_t* q, const uint8_t* q_scale, int64_t blocks32, bool nvfp4,
                          const float* tensor_scale, void* out, bool out_bf16, hipStream_t stream) {
  const unsigned grid = (unsigned)cdiv(blocks32, 256);
  if (out_bf16) {
    if (nvfp4) dequantise_kernel<true, true><<<grid, 256, 0, stream>>>(q, q_scale, blocks32, tensor_scale, out);
    else dequantise_kernel<true, false><<<grid, 256, 0, stream>>>(q, q_scale, blocks32, tensor_scale, out);
  } else {
    if (nvfp4) dequantise_kernel<false, true><<<grid, 256, 0, stream>>>(q, q_scale, blocks32, tensor_scale, out);
    else dequantise_kernel<false, false><<<grid, 256, 0, stream>>>(q, q_scale, blocks32, tensor_scale, out);
  }
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_nvfp4_tensor_scale(const void* x, bool bf16, int64_t n16, float* scale, uint32_t* partial, hipStream_t stream) {
  const int blocks = (int)min(cdiv(n16, 512 * 4), (int64_t)kAmaxBlocks);
  const u4v* p = static_cast<const u4v*>(x);
  if (bf16) amax_kernel<true><<<blocks, 512, 0, stream>>>(p, n16, partial, scale);
  else amax_kernel<false><<<blocks, 512, 0, stream>>>(p, n16, partial, scale);
  if (blocks > 1) amax_finish_kernel<<<1, 512, 0, stream>>>(partial, blocks, scale);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace mxf
