// Low-rank adapters of many requests beside one shared FP4 projection:
//   c[t] = a[t] . W_hat^T + scaling[l] * (a[t] . lora_a[l]^T) . lora_b[l]^T
// with l = seg_adapter[s] of the segment s that holds row t (negative: no adapter).
//   shrink:  low[t] = scaling[l] * a[t] . lora_a[l]^T, fp32, K split over the waves of a
//            workgroup (and over workgroups when rows are few: slices, summed by the reader)
//   M > 64:  the tiled product of w4a16_tile.hip takes low . lora_b^T into its
//            accumulators after the last stage, so c is written once
//   M <= 64: the weight-streaming product of gemm_w4a16.hip leaves its K slices in the
//            workspace; one pass adds them, the slices of low and the fp32 expansion.
#include "w4a16_tile.hpp"

namespace mxf {

namespace {

struct ShrinkArgs {
  const uint16_t* a;
  const uint16_t* lora_a;
  const float* scaling;
  const int32_t* seg_off;
  const int32_t* seg_adapter;
  float* low;
  int64_t M, K;
  int rank, L, S, zsplit;
};

// first segment s with seg_off[s + 1] > t (S if none), by halving
__device__ __forceinline__ int segment_of(const int32_t* __restrict__ seg_off, int S, int64_t t) {
  int lo = 0, hi = S;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if ((int64_t)seg_off[mid + 1] > t) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// Workgroup (x, y, z): rows [16 x, 16 x + 16), K slice y, every zsplit-th segment of those
// rows from the z-th on. 8 waves split the slice's K; RF fragments of 16 ranks.
template <int RF>
__global__ void __launch_bounds__(512) lora_shrink_kernel(ShrinkArgs p) {
  __shared__ float part[8][RF * 4 * 64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, g = lane >> 4, r16 = lane & 15;
  const int64_t K = p.K, row0 = (int64_t)blockIdx.x * 16, row1 = min(row0 + 16, p.M);
  const int nk = (int)(K / 32), ns = (int)gridDim.y * 8, me = (int)blockIdx.y * 8 + wave;
  const int k0 = (int)((int64_t)me * nk / ns), k1 = (int)((int64_t)(me + 1) * nk / ns);
  const uint16_t* const ap = p.a + min(row0 + r16, p.M - 1) * K + 8 * g;
  for (int s = segment_of(p.seg_off, p.S, row0) + (int)blockIdx.z; s < p.S; s += p.zsplit) {
    const int64_t lo = max((int64_t)p.seg_off[s], row0), hi = min((int64_t)p.seg_off[s + 1], row1);
    if ((int64_t)p.seg_off[s] >= row1) break;
    const int l = p.seg_adapter[s];
    if (l < 0 || l >= p.L || hi <= lo) continue;
    const uint16_t* bp[RF];
#pragma unroll
    for (int f = 0; f < RF; ++f) bp[f] = p.lora_a + ((int64_t)l * p.rank + min(16 * f + r16, p.rank - 1)) * K + 8 * g;
    v4f acc[RF];
#pragma unroll
    for (int f = 0; f < RF; ++f) acc[f] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int k = k0; k < k1; ++k) {
      const v8bf x = __builtin_bit_cast(v8bf, *reinterpret_cast<const v4i*>(ap + 32 * k));
#pragma unroll
      for (int f = 0; f < RF; ++f) {
        const v8bf w = __builtin_bit_cast(v8bf, *reinterpret_cast<const v4i*>(bp[f] + 32 * k));
        acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, w, acc[f], 0, 0, 0);
      }
    }
    __syncthreads();  // the previous segment's sums have been read
#pragma unroll
    for (int f = 0; f < RF; ++f)
#pragma unroll
      for (int v = 0; v < 4; ++v) part[wave][(4 * f + v) * 64 + lane] = acc[f][v];
    __syncthreads();
    const float scale = p.scaling[l];
    for (int i = wave; i < 4 * RF; i += 8) {
      float t = 0.0f;
#pragma unroll
      for (int w = 0; w < 8; ++w) t += part[w][i * 64 + lane];
      const int64_t row = row0 + 4 * g + (i & 3);
      const int r = 16 * (i >> 2) + r16;
      if (row >= lo && row < hi && r < p.rank)
        p.low[((int64_t)blockIdx.y * p.M + row) * p.rank + r] = scale * t;
    }
  }
}

struct FinishArgs {
  const float* base;  // [bslices][M][N]
  const float* low;   // [lslices][M][rank]
  const uint16_t* lora_b;
  const int32_t* seg_off;
  const int32_t* seg_adapter;
  void* out;
  int64_t M, N;
  int bslices, lslices, rank, L, S;
};

// one row, 256 columns per workgroup of one wave: 4 columns per lane
template <bool kOutBF16>
__global__ void __launch_bounds__(64) lora_finish_kernel(FinishArgs p) {
  __shared__ float low[128];
  const int64_t t = blockIdx.y;
  const int64_t n = (int64_t)blockIdx.x * 256 + 4 * threadIdx.x;
  const int s = segment_of(p.seg_off, p.S, t);
  int l = -1;
  if (s < p.S && (int64_t)p.seg_off[s] <= t) l = p.seg_adapter[s];
  const bool has = l >= 0 && l < p.L;
  if (has)
    for (int r = threadIdx.x; r < p.rank; r += 64) {
      float v = 0.0f;
      for (int i = 0; i < p.lslices; ++i) v += p.low[((int64_t)i * p.M + t) * p.rank + r];
      low[r] = v;
    }
  __syncthreads();
  if (n >= p.N) return;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < p.bslices; ++i) {
    const float4 u = *reinterpret_cast<const float4*>(p.base + ((int64_t)i * p.M + t) * p.N + n);
    v[0] += u.x, v[1] += u.y, v[2] += u.z, v[3] += u.w;
  }
  if (has) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint16_t* b = p.lora_b + ((int64_t)l * p.N + n + c) * p.rank;
      float d = 0.0f;
      for (int r = 0; r < p.rank; r += 8) {
        const v4i w = *reinterpret_cast<const v4i*>(b + r);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          d = fmaf(low[r + 2 * i], __uint_as_float((uint32_t)w[i] << 16), d);
          d = fmaf(low[r + 2 * i + 1], __uint_as_float((uint32_t)w[i] & 0xFFFF0000u), d);
        }
      }
      v[c] += d;
    }
  }
  const int64_t at = t * p.N + n;
  if (kOutBF16)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) =
        make_uint2(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]));
  else *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(v[0], v[1], v[2], v[3]);
}

}  // namespace

int lora_shrink_slices(int64_t M, int64_t K) {
  // few rows: K in slices of about 1024 so that more compute units load
  return M > 64 ? 1 : (int)(K / 1024 < 1 ? 1 : K / 1024);
}

int lora_base_slices(int64_t M, int64_t N, int64_t K) { return M <= 64 ? w4a16_ksplit(M, N, K) : 0; }

int launch_w16_lora(const W16LoraArgs& p, bool nv, bool out_bf16, hipStream_t stream) {
  const int ls = lora_shrink_slices(p.M, p.K);
  float* const base = p.workspace;
  float* const low = base + (int64_t)lora_base_slices(p.M, p.N, p.K) * p.M * p.N;
  if (p.S > 0) {
    const int64_t blocks = cdiv(p.M, 16);
    const int64_t z = cdiv(p.S, blocks) < 16 ? cdiv(p.S, blocks) : 16;
    ShrinkArgs s{p.a, p.lora_a, p.scaling, p.seg_off, p.seg_adapter, low, p.M, p.K, p.rank, p.L, p.S, (int)z};
    const dim3 grid((unsigned)blocks, (unsigned)ls, (unsigned)z);
    if (p.rank <= 16) lora_shrink_kernel<1><<<grid, 512, 0, stream>>>(s);
    else if (p.rank <= 32) lora_shrink_kernel<2><<<grid, 512, 0, stream>>>(s);
    else if (p.rank <= 64) lora_shrink_kernel<4><<<grid, 512, 0, stream>>>(s);
    else lora_shrink_kernel<8><<<grid, 512, 0, stream>>>(s);
  }
  if (p.M > 64) {
    W16TileArgs a{};
    a.a = p.a;
    a.a_rows = a.R = p.M;
    a.topk = a.E = 1;
    a.w = p.w;
    a.ws = p.ws;
    a.N = p.N;
    a.K = p.K;
    a.out = p.out;
    a.low = low;
    a.nslice = ls;
    a.rank = p.rank;
    a.L = p.L;
    a.S = p.S;
    a.seg_off = p.seg_off;
    a.seg_adapter = p.seg_adapter;
    a.lora_b = p.lora_b;
    launch_w16_tile_lora(a, nv, out_bf16, stream);
  } else {
    launch_w4a16_slices(nv, p.a, p.M, p.N, p.K, p.w, p.ws, base, stream);
    FinishArgs f{base, low, p.lora_b, p.seg_off, p.seg_adapter, p.out, p.M, p.N, lora_base_slices(p.M, p.N, p.K),
                 ls, p.rank, p.L, p.S};
    const dim3 grid((unsigned)cdiv(p.N, 256), (unsigned)p.M);
    if (out_bf16) lora_finish_kernel<true><<<grid, 64, 0, stream>>>(f);
    else lora_finish_kernel<false><<<grid, 64, 0, stream>>>(f);
  }
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace mxf
