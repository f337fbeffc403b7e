// The product of two quantised matrices: C[M][N] = g_a g_b A_hat B_hat^T, both operands 4-bit codes
// with block scales, K contiguous (fp4_gemm).
//
// MXFP4: codes and scales go into the scaled MFMA as they are (32x32x64, one 32-block a lane).
// NVFP4: that instruction knows no UE4M3 scales of 16, so a lane turns its 32 codes into fp16
// (code x scale has at most 6 significant bits and lies in 2^-10 .. 2688: exact) in front of four
// 32x32x16 fp16 MFMAs. Both take the same 16 bytes of a row per lane and 64 k, so copies, LDS layout
// and epilogue are one.
//
// A workgroup computes BM x BN with WM x WN waves of 32 FM x 32 FN; B is the MFMA's first operand, so
// that a lane ends up with runs of 4 consecutive columns of one row. Two LDS slots of 256 k (128 bytes
// a row, 16-byte chunks XOR-swizzled by the row): the copies of stage st + 1 go out at the top of
// stage st and land while it is computed. MFMA step s of a stage takes, in lane group g (lane / 32),
// the 32-block 4 g + s of both operands. Scales come in groups of 32 bytes a row (1024 k of MXFP4, 512 k of NVFP4).
//
// What bounds it (256 x 256 tiles). NVFP4, 4096 x 4096 x 7168: 186-199 us by the card = 1.2-1.3 PFLOP/s, the
// rate of a library's bf16 product of that size (188 us): the MFMA busy 56 to 59 % at the 1.7 to 1.9 GHz that the power
// leaves. Smaller tiles share a decoded operand among fewer MFMAs: with 128 x 128 the vector unit
// (8 instructions for 8 codes) has as much to do as the MFMA. MXFP4, 4096 x 7168 x 16384: 250-262 us = 3.7-3.8
// PFLOP/s, the MFMA busy 47 % at 1.95 GHz; without its copies the kernel takes 92 % of that time, the copies alone 77 %.
// Not faster: 4 waves of 128 x 128 (NVFP4 as fast, MXFP4 4 to 8 % slower), the first fragments of a stage
// read before the last step of the one before (NVFP4 2 % faster, MXFP4 5 % slower), 128 x 256 tiles, wave priorities.
//
// K need not be a multiple of 256: in the last stage's missing half (lane group 1) both scales are
// taken as zero bytes (2^-127 or 0), which leaves products of at most 36 x 2^-254: nothing in fp32.
// Rows past M or N read as zeros through the range-checked resources and are not stored.
#pragma once

#include "fp4_pair_plan.hpp"
#include "w4a16_common.hpp"
#include "w4a16_plan.hpp"

namespace mxf {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

struct Fp4PairArgs {
  const uint8_t *a, *as, *b, *bs;
  const float *ga, *gb;  // scales of the tensors (null: 1)
  void* out;             // [M][N], or the K slices' sums [slices][M][N] fp32
  int64_t M, N, K;
  int slices;
};

__device__ __forceinline__ v16f mfma32x32x16h(v8h a, v8h b, v16f c) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
#else
  return c;
#endif
}

// two UE4M3 bytes (the low or high half of a dword) -> fp16, exact
template <bool kHigh>
__device__ __forceinline__ v2h scales_to_half(uint32_t w) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.0f, kHigh);
#else
  return v2h{};
#endif
}

// 8 codes x a scale -> 8 fp16, exact
__device__ __forceinline__ v8h decode8_half(uint32_t codes, _Float16 scale) {
#if defined(__HIP_DEVICE_COMPILE__)
  const v2h s = {scale, scale};
  const v2h p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 0) * s;
  const v2h p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 1) * s;
  const v2h p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 2) * s;
  const v2h p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 3) * s;
  return v8h{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
#else
  return v8h{};
#endif
}

// x g_a g_b (null: 1). Either scale may lie at an end of fp32's range, so their mantissas are multiplied first and the
// exponents are applied together: x, a sum of products of 2^-20 and more, keeps its bits, whichever operand has which
struct PairScale {
  float m;
  int e;
  __device__ __forceinline__ PairScale(const float* ga, const float* gb) : m(1.0f), e(0) {
    int i;
    if (ga) {
      m = frexpf(*ga, &i);
      e = i;
    }
    if (gb) {
      m *= frexpf(*gb, &i);
      e += i;
    }
  }
  __device__ __forceinline__ float operator()(float x) const { return ldexpf(x * m, e); }
};

template <int BM, int BN>
struct alignas(16) Fp4PairRing {
  uint8_t SA[2][BM * 32], SB[2][BN * 32];
  uint8_t A[2][BM * 128], B[2][BN * 128];
};

template <int BM, int BN, int WM, int WN, bool kNV, bool kOutBF16, bool kSlices>
__global__ void __launch_bounds__(64 * WM * WN) fp4_pair_kernel(Fp4PairArgs a) {
  constexpr int NW = WM * WN, FM = BM / WM / 32, FN = BN / WN / 32;
  constexpr int IA = BM * 8 / 64 / NW, IB = BN * 8 / 64 / NW;  // 16-byte copies a lane and stage
  constexpr int ISA = BM * 2 / 64, ISB = BN * 2 / 64;          // of a scale group, in all
  constexpr int G = pair_group_stages(kNV);                    // stages of a scale group
  constexpr int IS = (ISA + ISB + NW - 1) / NW;                // of them a wave: A's, then B's
  static_assert(IA >= 1 && IB >= 1, "tile shape");
  __shared__ Fp4PairRing<BM, BN> ring;
  static_assert(sizeof(ring) <= 160 * 1024 && sizeof(ring) >= NW * 8192, "LDS");

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, g = lane >> 5,
            r32 = lane & 31;
  const int wm = wave / WN, wn = wave % WN;
  const int64_t M = a.M, N = a.N, K = a.K, wrow = K / 2, srow = K / (kNV ? 16 : 32);
  const uint32_t units = (uint32_t)((M + BM - 1) / BM), ntiles = (uint32_t)((N + BN - 1) / BN);
  uint32_t w;
  if (!w16_range(units * ntiles, (int)(blockIdx.x & 7u), (int)(blockIdx.x >> 3), w)) return;
  int n_tile, unit;
  w16_place(w, units, ntiles, n_tile, unit);
  const int64_t row0 = (int64_t)unit * BM, col0 = (int64_t)n_tile * BN;
  const int m = (int)min((int64_t)BM, M - row0), n = (int)min((int64_t)BN, N - col0);
  const uint32_t stages = (uint32_t)((K + 255) / 256);
  const int st0 = kSlices ? (int)w16_share(stages, (int)blockIdx.y, a.slices) : 0;
  const int nst = kSlices ? (int)w16_share(stages, (int)blockIdx.y + 1, a.slices) : (int)stages;

  const buf_rsrc ra = make_rsrc(a.a + row0 * wrow, (uint32_t)(m * wrow));
  const buf_rsrc ras = make_rsrc(a.as + row0 * srow, (uint32_t)(m * srow));
  const buf_rsrc rb = make_rsrc(a.b + col0 * wrow, (uint32_t)(n * wrow));
  const buf_rsrc rbs = make_rsrc(a.bs + col0 * srow, (uint32_t)(n * srow));
  uint32_t va[IA], vb[IB], vs[IS];
#pragma unroll
  for (int q = 0; q < IA; ++q) {
    va[q] = (uint32_t)pair_copy_from((wave * IA + q) * 64 + lane, wrow);
  }
#pragma unroll
  for (int q = 0; q < IB; ++q) {
    vb[q] = (uint32_t)pair_copy_from((wave * IB + q) * 64 + lane, wrow);
  }
#pragma unroll
  for (int q = 0; q < IS; ++q) {
    const int p = wave + NW * q;
    vs[q] = (uint32_t)pair_scales_from(p < ISA ? p : p - ISA, lane, srow);
  }
  auto issue = [&](int slot, int st) {
#pragma unroll
    for (int q = 0; q < IA; ++q) buf_dma16(ra, &ring.A[slot][(wave * IA + q) * 1024], va[q], (uint32_t)st * 128);
#pragma unroll
    for (int q = 0; q < IB; ++q) buf_dma16(rb, &ring.B[slot][(wave * IB + q) * 1024], vb[q], (uint32_t)st * 128);
  };
  auto issue_scales = [&](int grp) {
#pragma unroll
    for (int q = 0; q < IS; ++q) {
      const int p = wave + NW * q;
      if (p < ISA) buf_dma16(ras, &ring.SA[grp & 1][p * 1024], vs[q], (uint32_t)grp * 32);
      else if (p < ISA + ISB) buf_dma16(rbs, &ring.SB[grp & 1][(p - ISA) * 1024], vs[q], (uint32_t)grp * 32);
    }
  };
  issue_scales(st0 / G);
  issue(0, st0);
  const PairScale scale(kNV && !kSlices ? a.ga : nullptr, kNV && !kSlices ? a.gb : nullptr);  // MXFP4 has none

  v16f acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int f = 0; f < FN; ++f) acc[i][f] = v16f{};
  int arow[FM], brow[FN], aoff[FM], boff[FN];
#pragma unroll
  for (int f = 0; f < FM; ++f) {
    arow[f] = 32 * (FM * wm + f) + r32;
    aoff[f] = pair_block_at(arow[f], g);
  }
#pragma unroll
  for (int f = 0; f < FN; ++f) {
    brow[f] = 32 * (FN * wn + f) + r32;
    boff[f] = pair_block_at(brow[f], g);
  }

  struct Frags {
    v4i a[FM], b[FN];
  };
  auto compute = [&](const uint8_t* As, const uint8_t* Bs, int st) __attribute__((always_inline)) {
    constexpr int W = pair_scale_words(kNV);
    uint32_t sa[FM][W], sb[FN][W];
    const uint8_t* const SAs = &ring.SA[(st / G) & 1][pair_scales_at(st, g, kNV)];
    const uint8_t* const SBs = &ring.SB[(st / G) & 1][pair_scales_at(st, g, kNV)];
    const bool past = pair_past(g, st, K);
#pragma unroll
    for (int i = 0; i < W; ++i) {
#pragma unroll
      for (int f = 0; f < FM; ++f) {
        sa[f][i] = *reinterpret_cast<const uint32_t*>(SAs + pair_scales_row(32 * (FM * wm + f) + r32) + 4 * i);
        if (past) sa[f][i] = 0;
      }
#pragma unroll
      for (int f = 0; f < FN; ++f) {
        sb[f][i] = *reinterpret_cast<const uint32_t*>(SBs + pair_scales_row(32 * (FN * wn + f) + r32) + 4 * i);
        if (past) sb[f][i] = 0;
      }
    }
    auto load = [&](int s, Frags& F) __attribute__((always_inline)) {
#pragma unroll
      for (int f = 0; f < FM; ++f) {
        int o = aoff[f];
        asm volatile("" : "+v"(o));
        F.a[f] = *reinterpret_cast<const v4i*>(As + pair_step(o, s));
      }
#pragma unroll
      for (int f = 0; f < FN; ++f) {
        int o = boff[f];
        asm volatile("" : "+v"(o));
        F.b[f] = *reinterpret_cast<const v4i*>(Bs + pair_step(o, s));
      }
    };
    Frags F[2];
    load(0, F[0]);
    static_for<0, 4>([&](auto S_) __attribute__((always_inline)) {
      constexpr int s = decltype(S_)::value;
      if constexpr (s < 3) load(s + 1, F[(s + 1) & 1]);
      const Frags& f = F[s & 1];
      if constexpr (kNV) {
        v2h ha[FM], hb[FN];
#pragma unroll
        for (int i = 0; i < FM; ++i) ha[i] = scales_to_half<(s & 1) != 0>(sa[i][s / 2]);
#pragma unroll
        for (int i = 0; i < FN; ++i) hb[i] = scales_to_half<(s & 1) != 0>(sb[i][s / 2]);
static_for<0, 4>([&](auto J_) __attribute__((always_inline)) {
          constexpr int j = decltype(J_)::value;
          v8h av[FM];
#pragma unroll
          for (int i = 0; i < FM; ++i) av[i] = decode8_half((uint32_t)f.a[i][j], ha[i][j / 2]);
#pragma unroll
          for (int k = 0; k < FN; ++k) {
            const v8h bv = decode8_half((uint32_t)f.b[k][j], hb[k][j / 2]);
#pragma unroll
            for (int i = 0; i < FM; ++i) acc[i][k] = mfma32x32x16h(bv, av[i], acc[i][k]);
          }
        });
      } else {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int k = 0; k < FN; ++k)
            acc[i][k] = mfma32x32x64<kFmtFP4, kFmtFP4, s>(v8i{f.b[k][0], f.b[k][1], f.b[k][2], f.b[k][3], 0, 0, 0, 0},
                                                          v8i{f.a[i][0], f.a[i][1], f.a[i][2], f.a[i][3], 0, 0, 0, 0},
                                                          acc[i][k], (int)sb[k][0], (int)sa[i][0]);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  const bool active = 32 * FM * wm < m && 32 * FN * wn < n;
  // stage st: its copies are the only ones in flight; the barrier also means that every wave is done
  // with stage st - 1, whose slot (and scale group) the next copies fill
  auto step = [&](auto I, int st) __attribute__((always_inline)) {
    constexpr int i = decltype(I)::value;
    wait_vmcnt<0>();
    lds_barrier();
    if (st + 1 < nst) issue(i ^ 1, st + 1);
    if (w16_begins_scales(st, st0, G, nst)) issue_scales(st / G + 1);
    __builtin_amdgcn_sched_barrier(0);
    if (active) compute(ring.A[i], ring.B[i], st);
  };
  for (int st = st0; st < nst; st += 2) {
    step(std::integral_constant<int, 0>{}, st);
    if (st + 1 < nst) step(std::integral_constant<int, 1>{}, st + 1);
  }
  lds_barrier();  // every wave is done with the ring
  if (!active) return;

  // epilogue: 32 rows x PF fragments at a time through the wave's 8 KB of the ring (runs of 4 columns
  // in, 16-byte pieces of whole row segments out)
  constexpr int ES = kOutBF16 ? 2 : 4, PF = FN * 32 * ES > 256 ? 256 / (32 * ES) : FN;
  constexpr int NCH = PF * 32 * ES / 16;
  static_assert(FN % PF == 0 && 32 * 16 * NCH <= 8192, "passes");
  uint8_t* const stg = reinterpret_cast<uint8_t*>(&ring) + wave * 8192;
  uint8_t* const out = static_cast<uint8_t*>(a.out) + (kSlices ? (int64_t)blockIdx.y * M * N * 4 : 0);
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int p = 0; p < FN / PF; ++p) {
#pragma unroll
      for (int f = 0; f < PF; ++f)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v[k] = acc[i][p * PF + f][4 * j + k];
            if constexpr (kNV && !kSlices) v[k] = scale(v[k]);
          }
          if (kOutBF16) {
            *reinterpret_cast<uint2*>(stg + pair_out_to(f, j, g, r32, ES, NCH)) =
                make_uint2(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]));
          } else {
            *reinterpret_cast<float4*>(stg + pair_out_to(f, j, g, r32, ES, NCH)) = make_float4(v[0], v[1], v[2], v[3]);
          }
        }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
      for (int k = 0; k < NCH / 2; ++k) {
        const int idx = lane + 64 * k, rr = idx / NCH, c = idx % NCH;
        const v4i v = *reinterpret_cast<const v4i*>(stg + pair_out_from(rr, c, NCH));
        const int lrow = 32 * (FM * wm + i) + rr, lcol = 32 * (FN * wn + p * PF) + c * (16 / ES);
        if (lrow < m && lcol < n)
          __builtin_nontemporal_store(v, reinterpret_cast<v4i*>(out + ((row0 + lrow) * N + col0 + lcol) * ES));
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

}  // namespace mxf
