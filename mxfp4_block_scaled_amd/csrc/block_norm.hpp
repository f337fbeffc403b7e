// Block norm: what stands between two blocks of a decoder layer, in one pass over each row.
//   b = y_t, or sum_j expert_gates[t][j] * y[pair_row[t topk + j]] (the expert combine)
//   p = post_weight * b / sqrt(mean(b^2) + eps)        (or b)
//   r = residual_scale * x_t + gate * p
//   n = pre_weight * r / sqrt(mean(r^2) + eps), and its MX quantisation
// A workgroup owns one row; a thread owns C chunks of 8 consecutive columns and keeps
// them in fp32 registers from the first load to the last store, so every operand is read
// once and every result written once. HBM bound (latency bound for a few rows). The two
// mean squares are sums over the workgroup: butterfly inside a wave, then the waves'
// sums in wave order through LDS, so they do not depend on the run.
// What it measured (16384 x 7168, bf16, the combine of 6 rows, r and E4M3 out, 2.0 GB): 402 us
// with each operand loaded where it is used, 395 with x loaded beside y, 357 us = 5.6 TB/s with
// non-temporal loads of y and x and stores of r and n too (a batch this size passes through
// the caches only once; smaller ones keep theirs for the next operator). Walking several rows per
// workgroup with the weights in LDS and the next row loaded ahead was slower (456 us: half the
// waves). One chunk per thread instead of two for few rows: one row of 7168 4.5 us, 0.5 less, 64 rows
// with the combine 7.2 us, 1.2 less; for 4096 rows two chunks (55 against 66 us).
// Combines of 1 to 8 rows: 64 tokens 6.5 to 7.6 us, 16384 tokens 184, 207, 240, 279, 315, 357, 400,
// 452 us = 4.5 to 5.6 TB/s (one row after the other 195, 229, 264, 302, 343, -, 426, 467). All by
// replays of a captured graph.
// Roundings: everything is fp32 until each result is stored; n and the codes come from
// the unrounded r (not from its bf16 copy), the codes from the unrounded n.
#pragma once

#include "gemm_common.hpp"
#include "w4a16_plan.hpp"

namespace mxf {

namespace {

typedef unsigned int u4v __attribute__((ext_vector_type(4)));

template <bool kNT>
__device__ __forceinline__ u4v load16(const void* p) {
  const u4v* const q = static_cast<const u4v*>(p);
  if constexpr (kNT) return __builtin_nontemporal_load(q);
  else return *q;
}

template <bool kNT>
__device__ __forceinline__ void store16(void* p, u4v v) {
  if constexpr (kNT) __builtin_nontemporal_store(v, static_cast<u4v*>(p));
  else *static_cast<u4v*>(p) = v;
}

// 8 values as loaded: bf16 in raw[0], fp32 in both
struct Raw8 {
  u4v raw[2];
};

template <bool kNT>
__device__ __forceinline__ Raw8 load_raw8(const void* base, bool bf16, int64_t off) {
  Raw8 r;
  if (bf16) {
    r.raw[0] = load16<kNT>(static_cast<const uint16_t*>(base) + off);
  } else {
    r.raw[0] = load16<kNT>(static_cast<const float*>(base) + off);
    r.raw[1] = load16<kNT>(static_cast<const float*>(base) + off + 4);
  }
  return r;
}

__device__ __forceinline__ void unpack8(const Raw8& r, bool bf16, float (&v)[8]) {
  if (bf16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(r.raw[0][j] << 16);
      v[2 * j + 1] = __uint_as_float(r.raw[0][j] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = __uint_as_float(r.raw[0][j]);
      v[4 + j] = __uint_as_float(r.raw[1][j]);
    }
  }
}

template <bool kNT = false>
__device__ __forceinline__ void load8(const void* base, bool bf16, int64_t off, float (&v)[8]) {
  unpack8(load_raw8<kNT>(base, bf16, off), bf16, v);
}

template <bool kNT>
__device__ __forceinline__ void store8(void* base, bool bf16, int64_t off, const float (&v)[8]) {
  if (bf16) {
    u4v w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = bf16x2_bits(v[2 * j], v[2 * j + 1]);
    store16<kNT>(static_cast<uint16_t*>(base) + off, w);
  } else {
    float* const p = static_cast<float*>(base) + off;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u4v w;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = __float_as_uint(v[4 * h + j]);
      store16<kNT>(p + 4 * h, w);
    }
  }
}

// sum over the workgroup, the same in every thread; part holds one float per wave
__device__ __forceinline__ float block_sum(float v, float* part) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  const int nw = blockDim.x >> 6;
  if (nw == 1) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < nw; ++i) s += part[i];
  return s;
}

constexpr int64_t kFewRows = 256;
constexpr int64_t kOnce = int64_t(1) << 25;  // elements of a batch that the caches do not hold (64 MB in bf16)

// KT rows of y per token, 0: no combine. The rows' loads are in flight together (of rows wider than
// 32768 as many as the registers hold)
template <bool kYBF16, int KT, int C, bool kNT>
__global__ void __launch_bounds__(1024) block_norm_kernel(BlockNormArgs a) {
  __shared__ float part[2][16];
  const int64_t t = a.t0 + blockIdx.x;
  const int64_t H = a.H;
  const int tid = threadIdx.x, nt = blockDim.x;
  float v[C][8];
  bool ok[C];
  int64_t col[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    col[c] = 8 * (int64_t)(tid + c * nt);
    ok[c] = col[c] < H;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[c][i] = 0.0f;
  }
  // the block's output row, or the combine of the token's expert rows (slot order, fp32)
  if constexpr (KT == 0) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (ok[c]) load8<kNT>(a.y, kYBF16, t * H + col[c], v[c]);
  } else {
    constexpr int KM = C < 8 ? 8 : kYBF16 ? 4 : 2, KB = KT < KM ? KT : KM;
    int64_t row[KT];
    float g[KT];
    uint32_t keep[KT];
#pragma unroll
    for (int j = 0; j < KT; ++j) {
      row[j] = a.pair_row[t * KT + j];
      g[j] = a.expert_gates[t * KT + j];
      keep[j] = row[j] >= 0 && row[j] < a.y_rows ? ~0u : 0u;  // a dropped pair adds 0 times 0
      if (!keep[j]) row[j] = 0, g[j] = 0.0f;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (!ok[c]) continue;
#pragma unroll
      for (int b = 0; b < KT; b += KB) {
        Raw8 raw[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j)
          if (b + j < KT) raw[j] = load_raw8<kNT>(a.y, kYBF16, row[b + j] * H + col[c]);
#pragma unroll
        for (int j = 0; j < KB; ++j)
          if (b + j < KT) {
            float u[8];
#pragma unroll
            for (int h = 0; h < (kYBF16 ? 1 : 2); ++h) raw[j].raw[h] &= keep[b + j];
            unpack8(raw[j], kYBF16, u);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[c][i] = fmaf(g[b + j], u[i], v[c][i]);
          }
      }
    }
  }
  constexpr bool kEarlyX = KT > 0 && C <= 2;  // x on its way during the combine and the first mean
  Raw8 xr[C];
  if (kEarlyX && a.x) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (ok[c]) xr[c] = load_raw8<kNT>(a.x, a.x_bf16, t * H + col[c]);
  }
  if (a.post_weight) {
    float ss = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(v[c][i], v[c][i], ss);
    const float inv = rsqrtf(block_sum(ss, part[0]) / (float)H + a.eps);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (!ok[c]) continue;
      float w[8];
      load8(a.post_weight, a.weight_bf16, col[c], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] * inv * w[i];
    }
  }
  if (a.gate_mode != kGateNone) {
    float gt = 0.0f;
    if (a.gate_mode == kGateToken)
      gt = a.gate_bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.gate)[t] << 16)
                       : static_cast<const float*>(a.gate)[t];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (!ok[c]) continue;
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = gt;
      if (a.gate_mode == kGateChannel) load8(a.gate, a.gate_bf16, col[c], w);
      if (a.gate_mode == kGateFull) load8(a.gate, a.gate_bf16, t * H + col[c], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] *= w[i];
    }
  }
  if (a.x) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (!ok[c]) continue;
      float u[8];
      if constexpr (!kEarlyX) xr[c] = load_raw8<kNT>(a.x, a.x_bf16, t * H + col[c]);
      unpack8(xr[c], a.x_bf16, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = fmaf(a.residual_scale, u[i], v[c][i]);
    }
  }
  if (a.r) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (ok[c]) store8<kNT>(a.r, a.x_bf16, t * H + col[c], v[c]);
  }
  if (!a.n && !a.q) return;
  float ss = 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(v[c][i], v[c][i], ss);
  const float inv = rsqrtf(block_sum(ss, part[1]) / (float)H + a.eps);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (!ok[c]) continue;
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.0f;
    if (a.pre_weight) load8(a.pre_weight, a.weight_bf16, col[c], w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] * inv * w[i];
    if (a.n) store8<kNT>(a.n, a.n_bf16, t * H + col[c], v[c]);
  }
  if (!a.q) return;
  // a block of 32 columns is held by 4 neighbouring lanes (H % 32 == 0: all four or none)
#pragma unroll
  for (int c = 0; c < C; ++c) {
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(v[c][i]) & 0x7FFFFFFFu);
    amax = max(amax, (uint32_t)__shfl_xor((int)amax, 1));
    amax = max(amax, (uint32_t)__shfl_xor((int)amax, 2));
    if (!ok[c]) continue;
    const uint32_t byte = scale_byte_from_amax_bits(amax, a.q_fp4 ? kEmaxE2M1 : kEmaxE4M3);
    const float is = inv_scale_from_byte(byte);
    const int64_t at = t * H + col[c];
    if (a.q_fp4) {
      uint32_t w = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) w |= e2m1_code(v[c][i], is) << (4 * i);
      *reinterpret_cast<uint32_t*>(a.q + at / 2) = w;
    } else {
      uint32_t w[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i >> 2] |= e4m3_code(v[c][i], is) << (8 * (i & 3));
      *reinterpret_cast<uint2*>(a.q + at) = make_uint2(w[0], w[1]);
    }
    if ((tid & 3) == 0) a.q_scale[at / 32] = (uint8_t)byte;
  }
}

template <bool kYBF16, int KT, bool kNT>
void launch_c(BlockNormArgs a, hipStream_t stream) {
  // chunks of 8 columns per thread: one for few rows (the fewest steps of a row's latency), else
  // two while 1024 threads hold the row, more beyond
  const int64_t chunks = a.H / 8;
  const int C = chunks <= (a.T <= kFewRows ? 1024 : 64) ? 1 : chunks <= 2048 ? 2 : chunks <= 4096 ? 4 : 8;
  const dim3 block((unsigned)(cdiv(cdiv(chunks, C), 64) * 64));
  const int64_t most = kMaxThreads / block.x;  // rows of a launch
  for (a.t0 = 0; a.t0 < a.T; a.t0 += most) {
    const dim3 grid((unsigned)(a.T - a.t0 < most ? a.T - a.t0 : most));
    if (C == 1) block_norm_kernel<kYBF16, KT, 1, kNT><<<grid, block, 0, stream>>>(a);
    else if (C == 2) block_norm_kernel<kYBF16, KT, 2, kNT><<<grid, block, 0, stream>>>(a);
    else if (C == 4) block_norm_kernel<kYBF16, KT, 4, kNT><<<grid, block, 0, stream>>>(a);
    else block_norm_kernel<kYBF16, KT, 8, kNT><<<grid, block, 0, stream>>>(a);
  }
}

template <bool kYBF16, int KT>
void launch_nt(const BlockNormArgs& a, hipStream_t stream) {
  if (a.T * a.H >= kOnce) launch_c<kYBF16, KT, true>(a, stream);
  else launch_c<kYBF16, KT, false>(a, stream);
}

template <bool kYBF16, int KT>
void launch_k(const BlockNormArgs& a, hipStream_t stream) {
  if constexpr (KT < 8)
    if (a.topk > KT) return launch_k<kYBF16, KT + 1>(a, stream);
  launch_nt<kYBF16, KT>(a, stream);
}

}  // namespace

}  // namespace mxf
