// Launches of the product of two quantised matrices (fp4_pair.hpp) and the sum of its K slices.
#include "fp4_pair.hpp"
#include "launch.hpp"

namespace mxf {

namespace {

template <bool kOutBF16>
__global__ void __launch_bounds__(256) fp4_pair_sum_kernel(const float4* part, int slices, int64_t n4, const float* ga,
                                                           const float* gb, void* out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  float4 s = part[i];
  for (int k = 1; k < slices; ++k) {
    const float4 p = part[k * n4 + i];
    s.x += p.x;
    s.y += p.y;
    s.z += p.z;
    s.w += p.w;
  }
  const float x = ga ? *ga : 1.0f, y = gb ? *gb : 1.0f;
  s = make_float4(s.x * x * y, s.y * x * y, s.z * x * y, s.w * x * y);
  if (kOutBF16) static_cast<uint2*>(out)[i] = make_uint2(bf16x2_bits(s.x, s.y), bf16x2_bits(s.z, s.w));
  else static_cast<float4*>(out)[i] = s;
}

template <int BM, int BN, int WM, int WN, bool kNV>
void launch_tile(const Fp4PairArgs& a, bool out_bf16, hipStream_t stream) {
  const dim3 grid((unsigned)(8 * cdiv(cdiv(a.M, BM) * cdiv(a.N, BN), 8)), (unsigned)a.slices), threads(64 * WM * WN);
  if (a.slices > 1) fp4_pair_kernel<BM, BN, WM, WN, kNV, false, true><<<grid, threads, 0, stream>>>(a);
  else if (out_bf16) fp4_pair_kernel<BM, BN, WM, WN, kNV, true, false><<<grid, threads, 0, stream>>>(a);
  else fp4_pair_kernel<BM, BN, WM, WN, kNV, false, false><<<grid, threads, 0, stream>>>(a);
}

template <bool kNV>
void launch_plan(const Fp4PairPlan& p, const Fp4PairArgs& a, bool out_bf16, hipStream_t stream) {
  if (p.bm == 256) launch_tile<256, 256, 4, 2, kNV>(a, out_bf16, stream);
  else launch_tile<128, 128, 2, 2, kNV>(a, out_bf16, stream);
}

}  // namespace

size_t fp4_pair_workspace(int64_t M, int64_t N, int64_t K, bool nvfp4) {
  const Fp4PairPlan p = fp4_pair_plan(M, N, K, nvfp4);
  return p.slices > 1 ? (size_t)p.slices * (size_t)M * (size_t)N * sizeof(float) : 0;
}

int launch_fp4_pair(const uint8_t* a, const uint8_t* as, int64_t M, const uint8_t* b, const uint8_t* bs, int64_t N,
                    int64_t K, bool nvfp4, const float* ga, const float* gb, void* c, bool c_bf16, void* workspace,
                    hipStream_t stream) {
  const Fp4PairPlan p = fp4_pair_plan(M, N, K, nvfp4);
  const Fp4PairArgs args{a, as, b, bs, ga, gb, p.slices > 1 ? workspace : c, M, N, K, p.slices};
  if (nvfp4) launch_plan<true>(p, args, c_bf16, stream);
  else launch_plan<false>(p, args, c_bf16, stream);
  if (p.slices > 1) {
    const int64_t n4 = M * N / 4;
    const unsigned grid = (unsigned)cdiv(n4, 256);
    const float4* part = static_cast<const float4*>(workspace);
    if (c_bf16) fp4_pair_sum_kernel<true><<<grid, 256, 0, stream>>>(part, p.slices, n4, ga, gb, c);
    else fp4_pair_sum_kernel<false><<<grid, 256, 0, stream>>>(part, p.slices, n4, ga, gb, c);
  }
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace mxf
