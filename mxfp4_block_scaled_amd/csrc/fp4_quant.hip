// Quantisation of a matrix to 4-bit block formats and back.
//
// NVFP4: blocks of 16 with a UE4M3 scale s = E4M3(amax / (6 g)), g the tensor's scale (fp32);
// MXFP4: blocks of 32 with a UE8M0 scale 2^(floor(log2 amax) - 2), g = 1. An element's code is the
// E2M1 value nearest to x / d, d = s g (ties to even), or with random bytes r the upper of its two
// neighbours where the part above the lower one exceeds (r + 1/2) / 256. Blocks lie along the rows,
// along the columns (the codes of x^T, rows filled up to 128), or both from one read of x.
//
// x / d is the correctly rounded quotient: q = x (1/d) and one step with the exact remainder,
// q + (x - q d) (1/d). With the reciprocal alone a value halfway between two codes (often: x has 8
// bits and s 4) could land on either side of the tie.
//
// x once, the codes and scales once. Along rows HBM bounds it (4096 x 7168 bf16 14.2 us in MXFP4 and 15.9 in NVFP4, fp32 22
// and 24: 4.7 to 6 TB/s; stochastic 20 to 28, the random bytes with it); the stochastic choice in both directions the
// vector unit (bf16 to NVFP4 40 us, 1300 instructions for a lane's 32 values both ways are 30 of them; 53 with the choice
// by comparisons and the compiler's division). Where columns are wanted a workgroup holds a
// 128 x 128 tile of x in LDS; the codes along columns go back through LDS so that they leave as whole
// 64-byte pieces of a row of x^T.
#include "mx_codec.hpp"
#include "wave.hpp"
#include "w4a16_common.hpp"
#include "w4a16_plan.hpp"

namespace mxf {

namespace {

typedef unsigned int u4v __attribute__((ext_vector_type(4)));

constexpr float kTiny = 1.17549435e-38f;  // 2^-126

// 1 / v: the instruction is off by an ulp, one Newton step leaves half of one
__device__ __forceinline__ float reciprocal(float v) {
#if defined(__HIP_DEVICE_COMPILE__)
  const float r = __builtin_amdgcn_rcpf(v);
  return fmaf(fmaf(-v, r, 1.0f), r, r);
#else
  return 1.0f / v;
#endif
}

// x / d from r = 1 / d: one step with the exact remainder rounds it correctly (the sign of -0 is lost)
__device__ __forceinline__ float divide(float x, float d, float r) {
  const float q = x * r;
  return fmaf(fmaf(-q, d, x), r, q);
}

// what a matrix's block maxima are divided by: 6 g; both times a power of two where g lies so near an end of fp32's
// range that 6 g or its reciprocal would leave it
struct Top {
  float g, lift, six, inv;
  __device__ __forceinline__ explicit Top(const float* tensor_scale)
      : g(tensor_scale ? *tensor_scale : 1.0f),
        lift(g > 0x1p100f ? 0x1p-40f : g < 0x1p-80f ? 0x1p40f : 1.0f),
        six(6.0f * (g * lift)),
        inv(reciprocal(six)) {}
};

// what a block's elements are divided by
struct Divisor {
  float d, inv;
  uint32_t byte;
};

template <bool kNV>
__device__ __forceinline__ Divisor divisor_of(uint32_t amax_bits, const Top& top) {
  Divisor v;
  if (kNV) {
    v.byte = e4m3_mag_code(fminf(divide(__uint_as_float(amax_bits) * top.lift, top.six, top.inv), 448.0f));  // infinity gives NaN
    v.d = ue4m3_to_f32(v.byte) * top.g;
    const bool ok = v.d >= kTiny && v.d <= 3.0e38f;  // else the block is stored as zeros (g of no use, too)
    v.byte = ok ? v.byte : 0;
    v.d = ok ? v.d : 0.0f;
    v.inv = ok ? reciprocal(v.d) : 0.0f;
  } else {
    v.byte = scale_byte_from_amax_bits(amax_bits, kEmaxE2M1);
    v.d = ue8m0_to_f32(v.byte);
    v.inv = inv_scale_from_byte(min(v.byte, 253u));
  }
  return v;
}

// x / d, for the code nearest to it; or with a random byte r twice the value of the one of its two neighbours
// that r picks. With step the distance of the neighbours, u = |x / d| / step and t = (r + 1/2) / 256 that is
// ceil(u - t) steps: above floor(u) exactly if the part of u above it exceeds t. u - t is exact (t and u are
// multiples of u's last bit, or u < 1 and they are near each other or far from 0). Past 6 the conversion saturates.
template <bool kNV, bool kSR>
__device__ __forceinline__ float element(float x, uint32_t r, const Divisor& v) {
  const float q = kNV ? divide(x, v.d, v.inv) : x * v.inv;  // by a power of two: exact
  if constexpr (!kSR) return kNV ? copysignf(q, x) : q;
  const float t = fmaf((float)r, -1.0f / 256, -1.0f / 512);
  const uint32_t two = __float_as_uint(fmaxf(fabsf(q), 1.0f)) & 0x7F800000u;  // 2 step
  const float n = ceilf(fmaf(fabsf(q), __uint_as_float(0x7F800000u - two), t));
  return copysignf(n * __uint_as_float(two), x);
}

// 8 values -> one dword of codes
template <bool kSR>
__device__ __forceinline__ uint32_t pack8(const float (&x)[8]) {
  uint32_t w = 0;
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr float kScale = kSR ? 2.0f : 1.0f;  // element() has twice the value
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], kScale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], kScale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], kScale, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], kScale, 3);
#endif
  return w;
}

// A lane's part of a block: the 16 bytes that one load brings, 8 bf16 or 4 fp32 values, so that a wave's
// loads and stores are whole lines. The lanes of a block are neighbours and share its maximum.
template <bool kBF16>
constexpr int kPart = kBF16 ? 8 : 4;

template <bool kBF16>
__device__ __forceinline__ void part_values(const v4i& w, float (&x)[kPart<kBF16>]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (kBF16) {
      x[2 * j] = __uint_as_float((uint32_t)w[j] << 16);
      x[2 * j + 1] = __uint_as_float((uint32_t)w[j] & 0xFFFF0000u);
    } else {
      x[j] = __uint_as_float((uint32_t)w[j]);
    }
  }
}

// P values and random bytes (four a word) of a block -> P / 2 bytes of codes
template <bool kNV, bool kSR, int P>
__device__ __forceinline__ uint32_t codes_of(const float (&x)[P], const uint32_t* r, const Divisor& v) {
  float q[8] = {};
#pragma unroll
  for (int i = 0; i < P; ++i) q[i] = element<kNV, kSR>(x[i], kSR ? (r[i / 4] >> (8 * (i % 4))) & 0xFFu : 0, v);
  return pack8<kSR>(q);
}

template <int P>
__device__ __forceinline__ uint32_t amax_of(const float (&x)[P]) {
  float m = 0.0f;  // as floats: the magnitude is an operand's modifier, as integers an instruction
#pragma unroll
  for (int i = 0; i < P; ++i) m = fmaxf(m, fabsf(x[i]));
  return __float_as_uint(m);
}

template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_max(uint32_t m) {
#if defined(__HIP_DEVICE_COMPILE__)
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, kCtrl, 0xF, 0xF, true));
#endif
  return m;
}

// The part of a row's block that this lane holds: codes and, from the block's first lane, the scale.
// `at`: index of the part's first element in the matrix. All lanes of a block call this together.
template <bool kBF16, bool kNV, bool kSR>
__device__ __forceinline__ void quantise_part(const v4i& w, const uint32_t* r, const Top& top, int64_t at, bool in, uint8_t* q,
                                              uint8_t* q_scale) {
  constexpr int P = kPart<kBF16>, B = kNV ? 16 : 32, L = B / P;  // lanes of a block: 2, 4 or 8
  float x[P];
  part_values<kBF16>(w, x);
  uint32_t m = dpp_max<0xB1>(amax_of(x));       // lanes 1 0 3 2 of each four
  if constexpr (L >= 4) m = dpp_max<0x4E>(m);   // lanes 2 3 0 1
  if constexpr (L >= 8) m = dpp_max<0x141>(m);  // eight lanes mirrored
  const Divisor v = divisor_of<kNV>(m, top);
  const uint32_t c = codes_of<kNV, kSR>(x, r, v);
  if (!in) return;
  if constexpr (kBF16) *reinterpret_cast<uint32_t*>(q + at / 2) = c;
  else *reinterpret_cast<uint16_t*>(q + at / 2) = (uint16_t)c;
  if (at % B == 0) q_scale[at / B] = (uint8_t)v.byte;
}

// P bytes at a byte offset (out of range: zeros), four a word
template <int P>
__device__ __forceinline__ void load_dice(buf_rsrc rnd, uint32_t at, uint32_t (&r)[P / 4]) {
#if defined(__HIP_DEVICE_COMPILE__)
  if constexpr (P == 8) {
    const auto w = __builtin_amdgcn_raw_buffer_load_b64(rnd, (int)at, 0, 2);
    r[0] = w[0];
    r[1] = w[1];
  } else {
    r[0] = __builtin_amdgcn_raw_buffer_load_b32(rnd, (int)at, 0, 2);
  }
#endif
}

// Along rows only.
template <bool kBF16, bool kNV, bool kSR>
__global__ void __launch_bounds__(256) quantise_rows_kernel(Fp4QuantArgs a) {
  constexpr int P = kPart<kBF16>, U = 4;
  const int64_t first = (int64_t)blockIdx.x * (256 * U * P);  // element
  const Top top(a.tensor_scale);
  // past the matrix's end: zeros through the range-checked resources (a branch would wait for each load)
  const uint32_t n = (uint32_t)min(a.rows * a.cols - first, (int64_t)(256 * U * P));
  const buf_rsrc rx = make_rsrc(static_cast<const char*>(a.x) + first * (16 / P), n * (16 / P));
  const buf_rsrc rr = make_rsrc(kSR ? a.rnd + first : nullptr, kSR ? n : 0);
  v4i w[U];
  uint32_t r[U][P / 4] = {};
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const uint32_t i = threadIdx.x + 256 * k;
    w[k] = buf_load16_nt(rx, 16 * i, 0);
    if constexpr (kSR) load_dice<P>(rr, P * i, r[k]);
  }
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const uint32_t i = threadIdx.x + 256 * k;
    quantise_part<kBF16, kNV, kSR>(w[k], r[k], top, first + i * P, i * P < n, a.q, a.q_scale);
  }
}

// Along columns, and along rows where wanted: a 128 x 128 tile per workgroup. Workgroups of one XCD
// take neighbouring tiles, so that its L2 joins their pieces of the same lines.
template <bool kBF16, bool kNV, bool kSR>
__global__ void __launch_bounds__(512) quantise_both_kernel(Fp4QuantArgs a) {
  constexpr int P = kPart<kBF16>, B = kNV ? 16 : 32, T = 128, ES = kBF16 ? 2 : 4, RS = T * ES + 16;  // bytes of a row of the tile
  constexpr int C = kNV ? 2 : 1;           // columns of a lane
  constexpr int RP = 512 * P / T, U = T / RP;  // rows of a pass, passes
  __shared__ __align__(16) uint8_t tile[T * RS];
  __shared__ __align__(16) uint8_t dice[kSR ? T * T : 16];
  __shared__ __align__(16) uint32_t codes[T][T / 8 + 1];
  __shared__ uint8_t scales[T][T / B];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const uint32_t ct = (uint32_t)((a.cols + T - 1) / T), tiles = ct * (uint32_t)((a.rows + T - 1) / T);
  uint32_t t;
  if (!w16_range(tiles, (int)(blockIdx.x & 7u), (int)(blockIdx.x >> 3), t)) return;
  const int64_t row0 = (int64_t)(t / ct) * T, col0 = (int64_t)(t % ct) * T;
  const Top top(a.tensor_scale);

  const int c = tid % (T / P) * P, r0 = tid / (T / P);
  const int64_t col = col0 + c;
  // past the rows and columns: zeros through the range-checked resources (a branch would wait for each load)
  const uint32_t rows = (uint32_t)min(a.rows - row0, (int64_t)T), cols = (uint32_t)a.cols;
  const buf_rsrc rx = make_rsrc(static_cast<const char*>(a.x) + row0 * a.cols * ES, rows * cols * ES);
  const buf_rsrc rr = make_rsrc(kSR ? a.rnd + row0 * a.cols : nullptr, kSR ? rows * cols : 0);
  v4i w[U];
  uint32_t r[U][P / 4] = {};
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t at = (uint32_t)(RP * i + r0) * cols + (uint32_t)col;
    w[i] = buf_load16_nt(rx, col < a.cols ? at * ES : 0xFFFFFFF0u, 0);
    if constexpr (kSR) load_dice<P>(rr, col < a.cols ? at : 0xFFFFFFF0u, r[i]);
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int lr = RP * i + r0;
    *reinterpret_cast<v4i*>(tile + lr * RS + c * ES) = w[i];
    if constexpr (kSR) {
#pragma unroll
      for (int k = 0; k < P / 4; ++k) *reinterpret_cast<uint32_t*>(dice + lr * T + c + 4 * k) = r[i][k];
    }
  }
  if (a.q) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t row = row0 + RP * i + r0;
      quantise_part<kBF16, kNV, kSR>(w[i], r[i], top, row * a.cols + col, row < a.rows && col < a.cols, a.q, a.q_scale);
    }
  }
  __syncthreads();

  // columns: C of a lane, B rows at a time
  static_assert((T / B) * (T / (64 * C)) == 8, "a block of columns per wave");
  {
    const int i = wave % (T / B), c0 = (wave / (T / B)) * 64 * C + C * lane;
    float x[C][B];
    uint32_t dw[C][B / 4] = {};
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const uint8_t* at = tile + (B * i + k) * RS + c0 * ES;
      if constexpr (kBF16 && C == 2) {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(at);
        x[0][k] = __uint_as_float(v << 16);
        x[C - 1][k] = __uint_as_float(v & 0xFFFF0000u);
      } else {
#pragma unroll
        for (int h = 0; h < C; ++h)
          x[h][k] = kBF16 ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(at)[h] << 16)
                          : reinterpret_cast<const float*>(at)[h];
      }
      if constexpr (kSR) {
#pragma unroll
        for (int h = 0; h < C; ++h) dw[h][k / 4] |= (uint32_t)dice[(B * i + k) * T + c0 + h] << (8 * (k % 4));
      }
    }
#pragma unroll
    for (int h = 0; h < C; ++h) {
      const Divisor v = divisor_of<kNV>(amax_of(x[h]), top);
      scales[c0 + h][i] = (uint8_t)v.byte;
#pragma unroll
      for (int k = 0; k < B / 8; ++k) {
        float part[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) part[j] = x[h][8 * k + j];
        codes[c0 + h][B / 8 * i + k] = codes_of<kNV, kSR>(part, &dw[h][2 * k], v);
      }
    }
  }
  __syncthreads();

  // out: 64 bytes of codes and T / B scales of each column
  const int64_t padded = (a.rows + 127) / 128 * 128;
  const int oc = tid >> 2, p = tid & 3;
  if (col0 + oc < a.cols)
    *reinterpret_cast<uint4*>(a.qt + (col0 + oc) * (padded / 2) + row0 / 2 + 16 * p) =
        make_uint4(codes[oc][4 * p], codes[oc][4 * p + 1], codes[oc][4 * p + 2], codes[oc][4 * p + 3]);
  for (int idx = tid; idx < T * (T / B); idx += 512) {
    const int sc = idx / (T / B), k = idx % (T / B);
    if (col0 + sc < a.cols) a.qt_scale[(col0 + sc) * (padded / B) + row0 / B + k] = scales[sc][k];
  }
}

// 16 bytes of values a lane: 8 codes to bf16 or 4 to fp32, so that a wave stores whole lines
template <bool kBF16, bool kNV>
__global__ void __launch_bounds__(256) dequantise_kernel(const uint8_t* q, const uint8_t* q_scale, int64_t n,
                                                         const float* tensor_scale, void* out) {
  constexpr int P = kPart<kBF16>, B = kNV ? 16 : 32, U = 4;
  const int64_t i0 = (int64_t)blockIdx.x * (256 * U) + threadIdx.x;
  const float g = tensor_scale ? *tensor_scale : 1.0f;
  uint32_t w[U], b[U];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const int64_t i = min(i0 + 256 * k, n - 1);
    w[k] = kBF16 ? reinterpret_cast<const uint32_t*>(q)[i] : reinterpret_cast<const uint16_t*>(q)[i];
    b[k] = q_scale[i / (B / P)];
  }
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const int64_t i = i0 + 256 * k;
    if (i >= n) return;
    const float s = kNV ? ue4m3_to_f32(b[k] & 0x7Fu) : ue8m0_to_f32(b[k]);
    float v[8] = {};
#if defined(__HIP_DEVICE_COMPILE__)
    const v2f p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[k], 1.0f, 0);
    const v2f p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[k], 1.0f, 1);
    const v2f p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[k], 1.0f, 2);
    const v2f p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[k], 1.0f, 3);
    const float e[8] = {p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
#pragma unroll
    for (int j = 0; j < P; ++j) v[j] = e[j] * s * g;
#endif
    u4v d;
#pragma unroll
    for (int j = 0; j < 4; ++j) d[j] = kBF16 ? bf16x2_bits(v[2 * j], v[2 * j + 1]) : __float_as_uint(v[j]);
    __builtin_nontemporal_store(d, static_cast<u4v*>(out) + i);
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

// one wave, all of its loads in flight together
__global__ void __launch_bounds__(64) amax_finish_kernel(const uint32_t* partial, int n, float* scale) {
  uint32_t m[kAmaxBlocks / 64];
#pragma unroll
  for (int i = 0; i < kAmaxBlocks / 64; ++i) m[i] = partial[min((int)threadIdx.x + 64 * i, n - 1)];
#pragma unroll
  for (int i = 1; i < kAmaxBlocks / 64; ++i) m[0] = max(m[0], m[i]);
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) m[0] = max(m[0], (uint32_t)__shfl_xor((int)m[0], d));
  if (threadIdx.x == 0) *scale = scale_of_amax(m[0]);
}

template <bool kBF16, bool kNV, bool kSR>
void launch_quant_t(const Fp4QuantArgs& a, hipStream_t stream) {
  if (a.qt)
    quantise_both_kernel<kBF16, kNV, kSR><<<(unsigned)(8 * cdiv(cdiv(a.rows, 128) * cdiv(a.cols, 128), 8)), 512, 0, stream>>>(a);
  else
    quantise_rows_kernel<kBF16, kNV, kSR><<<(unsigned)cdiv(a.rows * a.cols / kPart<kBF16>, 1024), 256, 0, stream>>>(a);
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
  const int64_t n = blocks32 * (out_bf16 ? 4 : 8);
  const unsigned grid = (unsigned)cdiv(n, 1024);
  if (out_bf16) {
    if (nvfp4) dequantise_kernel<true, true><<<grid, 256, 0, stream>>>(q, q_scale, n, tensor_scale, out);
    else dequantise_kernel<true, false><<<grid, 256, 0, stream>>>(q, q_scale, n, tensor_scale, out);
  } else {
    if (nvfp4) dequantise_kernel<false, true><<<grid, 256, 0, stream>>>(q, q_scale, n, tensor_scale, out);
    else dequantise_kernel<false, false><<<grid, 256, 0, stream>>>(q, q_scale, n, tensor_scale, out);
  }
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

// Workgroups of the maximum of n16 16-byte pieces. One alone up to 256 KB: us a call, one launch | two,
// 64 KB 6.4 | 10.4, 256 KB 6.3 | 10.4; in a graph 3.0 | 4.3 and 5.5 | 4.3.
int amax_blocks(int64_t n16) {
  return n16 <= 16384 ? 1 : (int)min(cdiv(n16, 512 * 4), (int64_t)kAmaxBlocks);
}

int launch_nvfp4_tensor_scale(const void* x, bool bf16, int64_t n16, float* scale, uint32_t* partial, hipStream_t stream) {
  const int blocks = amax_blocks(n16);
  const u4v* p = static_cast<const u4v*>(x);
  if (bf16) amax_kernel<true><<<blocks, 512, 0, stream>>>(p, n16, partial, scale);
  else amax_kernel<false><<<blocks, 512, 0, stream>>>(p, n16, partial, scale);
  if (blocks > 1) amax_finish_kernel<<<1, 64, 0, stream>>>(partial, blocks, scale);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace mxf
