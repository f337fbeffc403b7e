// Backward pass of the gate-weighted combine out[t] = sum_j gates[t][j] y[pair_row[t topk + j]]:
//   dy[pair_row[p]] = gates[p] dout[t],   dgates[p] = sum_h dout[t][h] y[pair_row[p]][h]
// HBM-bound: every row of y is read once and every row of dy written once, whole lines at a time, and
// a token's row of dout is read once and kept in registers for its topk pairs. A pair's row is
// written by its own token alone, so nothing is added up in memory. 16384 x 7168 bf16, 6 rows each: 597-609 us
// for 3.06 GB = 5.0-5.1 TB/s, where a copy reaches 4.9.
#include "gemm_common.hpp"
#include "wave.hpp"

namespace mxf {

namespace {

// P consecutive values as they lie in memory: 16 bytes of the wider type, so that a wave's loads and
// stores are whole lines (4 fp32 values beside 4 bf16 ones of 8 bytes, or 8 bf16 ones)
template <bool kBF16, int P>
struct Part {
  static constexpr int W = kBF16 ? P / 2 : P;  // words
  typedef unsigned int Words __attribute__((ext_vector_type(W)));
  Words w;
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    w = __builtin_nontemporal_load(reinterpret_cast<const Words*>(static_cast<const char*>(p) + at * (kBF16 ? 2 : 4)));
  }
  __device__ __forceinline__ float get(int i) const {
    if (kBF16) return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    return __uint_as_float(w[i]);
  }
  __device__ static __forceinline__ void store(void* p, int64_t at, const float (&v)[P]) {
    Words d;
#pragma unroll
    for (int i = 0; i < W; ++i) d[i] = kBF16 ? bf16x2_bits(v[(2 * i) % P], v[(2 * i + 1) % P]) : __float_as_uint(v[i % P]);
    __builtin_nontemporal_store(d, reinterpret_cast<Words*>(static_cast<char*>(p) + at * (kBF16 ? 2 : 4)));
  }
};

constexpr int kChunks = 2;  // parts of a thread in a pass

// One workgroup per token and KJ of its pairs.
template <bool kYBF16, bool kDBF16, int KJ>
__global__ void __launch_bounds__(512) combine_backward_kernel(CombineBackwardArgs a) {
  constexpr int P = kYBF16 && kDBF16 ? 8 : 4;
  __shared__ float red[8][KJ];
  const int tid = threadIdx.x, nthr = blockDim.x, wave = tid >> 6, lane = tid & 63;
  const int parts = (a.topk + KJ - 1) / KJ;
  const int64_t t = blockIdx.x / parts;
  const int j0 = (int)(blockIdx.x % parts) * KJ;
  int64_t row[KJ];
  float g[KJ], dot[KJ];
#pragma unroll
  for (int j = 0; j < KJ; ++j) {
    const bool in = j0 + j < a.topk;
    const int64_t p = t * a.topk + (in ? j0 + j : 0);
    row[j] = in ? (int64_t)a.pair_row[p] : -1;
    if (row[j] >= a.y_rows) row[j] = -1;
    g[j] = a.gates[p];
    dot[j] = 0.0f;
  }
  for (int64_t c0 = 0; c0 < a.H; c0 += (int64_t)nthr * P * kChunks) {
    Part<kDBF16, P> d[kChunks];
    Part<kYBF16, P> y[KJ][kChunks];
    bool ok[kChunks];
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      const int64_t col = c0 + ((int64_t)k * nthr + tid) * P;
      ok[k] = col < a.H;
      if (!ok[k]) continue;
      d[k].load(a.dout, t * a.H + col);
      if (a.dgates) {
#pragma unroll
        for (int j = 0; j < KJ; ++j)
          if (row[j] >= 0) y[j][k].load(a.y, row[j] * a.H + col);
      }
    }
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      if (!ok[k]) continue;
      const int64_t col = c0 + ((int64_t)k * nthr + tid) * P;
      float dv[P];
#pragma unroll
      for (int i = 0; i < P; ++i) dv[i] = d[k].get(i);
#pragma unroll
      for (int j = 0; j < KJ; ++j) {
        if (row[j] < 0) continue;
        if (a.dgates) {
#pragma unroll
          for (int i = 0; i < P; ++i) dot[j] = fmaf(dv[i], y[j][k].get(i), dot[j]);
        }
        if (a.dy) {
          float v[P];
#pragma unroll
          for (int i = 0; i < P; ++i) v[i] = g[j] * dv[i];
          Part<kYBF16, P>::store(a.dy, row[j] * a.H + col, v);
        }
      }
    }
  }
  if (!a.dgates) return;
#pragma unroll
  for (int j = 0; j < KJ; ++j) {
    const float s = wave_sum(dot[j]);
    if (lane == 0) red[wave][j] = s;
  }
  __syncthreads();
  if (tid < KJ && j0 + tid < a.topk) {
    float s = 0.0f;
    for (int w = 0; w < nthr / 64; ++w) s += red[w][tid];
    a.dgates[t * a.topk + j0 + tid] = s;  // a dropped pair's sum is 0
  }
}

template <bool kYBF16, bool kDBF16>
void launch_t(const CombineBackwardArgs& a, int threads, hipStream_t stream) {
  const int kj = combine_backward_pairs(a.T, a.topk);
  const unsigned grid = (unsigned)(a.T * cdiv(a.topk, kj));
  switch (kj) {
    case 1: combine_backward_kernel<kYBF16, kDBF16, 1><<<grid, threads, 0, stream>>>(a); break;
    case 2: combine_backward_kernel<kYBF16, kDBF16, 2><<<grid, threads, 0, stream>>>(a); break;
    case 4: combine_backward_kernel<kYBF16, kDBF16, 4><<<grid, threads, 0, stream>>>(a); break;
    case 6: combine_backward_kernel<kYBF16, kDBF16, 6><<<grid, threads, 0, stream>>>(a); break;
    default: combine_backward_kernel<kYBF16, kDBF16, 8><<<grid, threads, 0, stream>>>(a); break;
  }
}

}  // namespace

// Pairs of a workgroup: all of a token's, so that dout is read once; one each while the tokens alone
// would leave compute units idle.
int combine_backward_pairs(int64_t T, int topk) {
  if (T < 256) return 1;
  return topk <= 2 ? topk : topk <= 4 ? 4 : topk <= 6 ? 6 : 8;
}

int combine_backward_threads(int64_t H, bool bf16) {
  return (int)min(cdiv(H, (bf16 ? 8 : 4) * kChunks * 64), (int64_t)8) * 64;
}

int launch_combine_backward(const CombineBackwardArgs& a, bool y_bf16, bool dout_bf16, hipStream_t stream) {
  const int threads = combine_backward_threads(a.H, y_bf16 && dout_bf16);
  if (y_bf16) {
    if (dout_bf16) launch_t<true, true>(a, threads, stream);
    else launch_t<true, false>(a, threads, stream);
  } else {
    if (dout_bf16) launch_t<false, true>(a, threads, stream);
    else launch_t<false, false>(a, threads, stream);
  }
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace mxf
