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
  if (ga || gb) {
    const PairScale scale(ga, gb);
    s = make_float4(scale(s.x), scale(s.y), scale(s.z), scale(s.w));
  }
  if (kOutBF16) static_cast<uint2*>(out)[i] = make_uint2(bf16x2_bits(s.x, s.y), bf16x2_bits(s.z, s.w));
  else static_cast<float4*>(out)[i] = s;
}

// Few tiles: 32 rows x 32 columns a workgroup, whose 8 waves share K. A wave copies its stages into two LDS
// slots of its own (whole lines, no barrier among waves) and the waves' sums meet in LDS: one launch, no
// workspace. The fixed order of the waves keeps results the same from run to run. 64 x 4096 x 7168: MXFP4
// 7.4 us, NVFP4 11 (its decoding takes the vector unit 3 us: 32 rows of A beside 32 of B). Loads straight
// into registers, a lane a row, cost the address unit 32 lines an instruction: 11 and 13 us, and the tiled
// kernel with K slices 19 and 22.
constexpr int kFewWaves = 8;
struct alignas(16) FewSlot {
  uint8_t A[32 * 128], B[32 * 128];
};

// a lane's scales of a stage, one load: 4 UE8M0 or 8 UE4M3 bytes
template <int W>
__device__ __forceinline__ void load_scales(buf_rsrc r, uint32_t voff, uint32_t soff, uint32_t (&s)[W]) {
#if defined(__HIP_DEVICE_COMPILE__)
  if constexpr (W == 2) {
    const auto w = __builtin_amdgcn_raw_buffer_load_b64(r, (int)voff, (int)soff, 0);
    s[0] = w[0];
    s[1] = w[1];
  } else {
    s[0] = __builtin_amdgcn_raw_buffer_load_b32(r, (int)voff, (int)soff, 0);
  }
#endif
}

template <bool kNV, bool kOutBF16>
__global__ void __launch_bounds__(64 * kFewWaves) fp4_few_kernel(Fp4PairArgs a) {
  constexpr int W = pair_scale_words(kNV);
  __shared__ union {
    FewSlot ring[kFewWaves][2];
    float part[kFewWaves][16 * 65];
  } lds;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, g = lane >> 5,
            r32 = lane & 31;
  const int64_t M = a.M, N = a.N, K = a.K, wrow = K / 2, srow = K / (kNV ? 16 : 32);
  const uint32_t ntiles = (uint32_t)((N + 31) / 32);
  const int64_t row0 = (int64_t)(blockIdx.x / ntiles) * 32, col0 = (int64_t)(blockIdx.x % ntiles) * 32;
  const int m = (int)min((int64_t)32, M - row0), n = (int)min((int64_t)32, N - col0);
  const uint32_t stages = (uint32_t)((K + 255) / 256);
  const int st0 = (int)w16_share(stages, wave, kFewWaves), nst = (int)w16_share(stages, wave + 1, kFewWaves);
  const buf_rsrc ra = make_rsrc(a.a + row0 * wrow, (uint32_t)(m * wrow));
  const buf_rsrc ras = make_rsrc(a.as + row0 * srow, (uint32_t)(m * srow));
  const buf_rsrc rb = make_rsrc(a.b + col0 * wrow, (uint32_t)(n * wrow));
  const buf_rsrc rbs = make_rsrc(a.bs + col0 * srow, (uint32_t)(n * srow));

  uint32_t at[4];  // row 8 q + lane / 8, 16-byte chunk lane % 8 of a stage
#pragma unroll
  for (int q = 0; q < 4; ++q) at[q] = (uint32_t)pair_copy_from(64 * q + lane, wrow);
  const uint32_t sat = pair_few_scales(r32, g, srow, kNV);
  struct Scales {
    uint32_t a[W], b[W];
  };
  auto issue = [&](FewSlot& slot, Scales& sc, int st) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      buf_dma16(rb, slot.B + 1024 * q, at[q], (uint32_t)st * 128);
      buf_dma16(ra, slot.A + 1024 * q, at[q], (uint32_t)st * 128);
    }
    __builtin_amdgcn_sched_barrier(0);  // the copies first: step() counts on it
    load_scales(rbs, sat, pair_few_scales_step(st, kNV), sc.b);
    load_scales(ras, sat, pair_few_scales_step(st, kNV), sc.a);
    __builtin_amdgcn_sched_barrier(0);
  };
  v16f acc = v16f{};
  auto compute = [&](const FewSlot& slot, Scales sc, int st) __attribute__((always_inline)) {
    if (pair_past(g, st, K)) {
#pragma unroll
      for (int k = 0; k < W; ++k) sc.a[k] = sc.b[k] = 0;
    }
    v4i fa[4], fb[4];
    const int o = pair_block_at(r32, g);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      fa[s] = *reinterpret_cast<const v4i*>(slot.A + pair_step(o, s));
      fb[s] = *reinterpret_cast<const v4i*>(slot.B + pair_step(o, s));
    }
    static_for<0, 4>([&](auto S_) __attribute__((always_inline)) {
      constexpr int s = decltype(S_)::value;
      if constexpr (kNV) {
        const v2h ha = scales_to_half<(s & 1) != 0>(sc.a[s / 2]), hb = scales_to_half<(s & 1) != 0>(sc.b[s / 2]);
        static_for<0, 4>([&](auto J_) __attribute__((always_inline)) {
          constexpr int j = decltype(J_)::value;
          acc = mfma32x32x16h(decode8_half((uint32_t)fb[s][j], hb[j / 2]), decode8_half((uint32_t)fa[s][j], ha[j / 2]), acc);
        });
      } else {
        acc = mfma32x32x64<kFmtFP4, kFmtFP4, s>(v8i{fb[s][0], fb[s][1], fb[s][2], fb[s][3], 0, 0, 0, 0},
                                                v8i{fa[s][0], fa[s][1], fa[s][2], fa[s][3], 0, 0, 0, 0}, acc,
                                                (int)sc.b[0], (int)sc.a[0]);
      }
    });
  };
  FewSlot* const slot = lds.ring[wave];
  Scales sc[2];
  // A stage's copies, then its loads; they return in order, so once at most those of the next stage are
  // outstanding the copies of this one have landed. No barrier: the slots are the wave's own.
  auto step = [&](auto I, int st) __attribute__((always_inline)) {
    constexpr int i = decltype(I)::value;
    if (st + 1 < nst) {
      issue(slot[i ^ 1], sc[i ^ 1], st + 1);
      wait_vmcnt<kFewCopies + kFewLoads>();
    } else {
      wait_vmcnt<0>();
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    compute(slot[i], sc[i], st);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  if (st0 < nst) issue(slot[0], sc[0], st0);
  const PairScale scale(kNV ? a.ga : nullptr, kNV ? a.gb : nullptr);
  for (int st = st0; st < nst; st += 2) {
    step(std::integral_constant<int, 0>{}, st);
    if (st + 1 < nst) step(std::integral_constant<int, 1>{}, st + 1);
  }
  __syncthreads();  // every wave is done with its slots
#pragma unroll
  for (int v = 0; v < 16; ++v) lds.part[wave][65 * v + lane] = acc[v];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 1024 / (64 * kFewWaves); ++k) {
    const int o = (int)threadIdx.x + 64 * kFewWaves * k, r = o >> 5, c = o & 31, from = pair_few_sum(r, c);
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) s += lds.part[w][from];
    if constexpr (kNV) s = scale(s);
    if (r >= m || c >= n) continue;
    if (kOutBF16) static_cast<__bf16*>(a.out)[(row0 + r) * N + col0 + c] = (__bf16)s;
    else static_cast<float*>(a.out)[(row0 + r) * N + col0 + c] = s;
  }
}

template <bool kNV>
void launch_few(const Fp4PairArgs& a, bool out_bf16, hipStream_t stream) {
  const unsigned grid = (unsigned)(cdiv(a.N, 32) * cdiv(a.M, 32));  // at most kMostFewTiles
  if (out_bf16) fp4_few_kernel<kNV, true><<<grid, 64 * kFewWaves, 0, stream>>>(a);
  else fp4_few_kernel<kNV, false><<<grid, 64 * kFewWaves, 0, stream>>>(a);
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
  if (p.bm == 32) launch_few<kNV>(a, out_bf16, stream);
  else if (p.bm == 256) launch_tile<256, 256, 4, 2, kNV>(a, out_bf16, stream);
  else if (p.bm == 64 && p.bn == 64) launch_tile<64, 64, 2, 2, kNV>(a, out_bf16, stream);
  else if (p.bm == 64) launch_tile<64, 128, 2, 2, kNV>(a, out_bf16, stream);
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
