// Tiled products of bf16 activations with FP4 weights: y = A . W_hat^T for many rows per
// weight matrix, either grouped by expert with ragged row ranges (moe_grouped_gemm_w4a16)
// or over one matrix with low-rank adapters beside it (fp4_gemm_w4a16_lora).
//
// A workgroup computes BM rows x BN weight rows with waves of 64 rows x 32 FN weight rows
// on the 32x32x16 bf16 MFMA (weights as the first operand, so a lane ends up with runs of
// 4 consecutive columns of one row). A stage is 64 k: BM x 128 bytes of activations,
// BN x 32 bytes of codes and one scale dword per weight row, all copied HBM -> LDS
// directly; three slots, the copies of stage st + 2 go out while st is computed. The
// weights stay 4 bits wide up to the registers: a lane reads the 16 bytes that hold 32
// codes of its weight row and converts 8 of them (exactly: a code times its scale has at
// most 5 significant bits) in front of each MFMA.
//
// K order: inside a stage MFMA j takes, in lane group g (lane / 32), k = 32 g + 8 j +
// [0, 8), for both operands: a weight lane's 16 bytes are 16-byte chunk g of its 32-byte
// stage row, one 32-element block, and an activation lane reads chunk 4 g + j of its
// 128-byte stage row. Chunks are XOR-swizzled per row so that the 16 lanes of an LDS
// cycle hit different banks.
//
// Rows past a unit's end and weight rows past N read as zero through the range-checked
// buffer resources and are not stored.
#include "w4a16_tile.hpp"

namespace mxf {

namespace {

template <int BM, int BN>
struct alignas(16) W16Slot {
  uint8_t A[BM * 128];
  uint8_t B[BN * 32];
  uint8_t Bs[BN * 4];
};
constexpr int kSlots = 3;

__device__ __forceinline__ int swz_a16(int r) { return (r & 7) ^ ((r >> 3) & 1); }  // 8 chunks per row
__device__ __forceinline__ int swz_b16(int r) { return (r >> 3) & 1; }              // 2 chunks per row

typedef short v8s __attribute__((ext_vector_type(8)));

__device__ __forceinline__ v16f mfma32x32x16(v8bf a, v8bf b, v16f c) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
#else
  (void)a;
  (void)b;
  return c;
#endif
}

// first segment s whose end seg_off[s + 1] lies past row t (S if none): 64 probes a step
__device__ __forceinline__ int first_segment(const int32_t* __restrict__ seg_off, int S, int64_t t) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = S;
  while (lo < hi) {
    const int step = (hi - lo + 63) / 64;
    const int64_t idx = lo + (int64_t)lane * step;
    const bool p = idx < hi && (int64_t)seg_off[idx < hi ? idx + 1 : 0] > t;
    const unsigned long long m = __ballot(p);
    const int probes = (hi - lo + step - 1) / step;
    const int f = m ? __ffsll((long long)m) - 1 : probes;  // the first probe past t
    const int nlo = f == 0 ? lo : lo + (f - 1) * step + 1;
    hi = f == probes ? hi : lo + f * step;
    lo = nlo;
    if (step == 1) break;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// BM x BN per workgroup of NW waves: BM / 64 waves over rows, the others over columns
template <int BM, int BN, int NW, bool kNV, bool kSwiglu, bool kOutBF16, bool kLora>
__global__ void __launch_bounds__(NW * 64) w16_tile_kernel(W16TileArgs a) {
  constexpr int WMN = BM / 64, WNN = NW / WMN, FN = BN / WNN / 32;
  constexpr int IA = BM * 8 / 64 / NW, IB = BN * 2 / 64 / NW;  // 16-byte copies per lane per stage
  static_assert(IA >= 1 && IB >= 1 && BN / 64 <= NW && (!kSwiglu || FN % 2 == 0), "tile shape");
  __shared__ W16Slot<BM, BN> ring[kSlots];
  static_assert(sizeof(ring) <= 160 * 1024 && sizeof(ring) >= NW * 8192, "the epilogue stages through the ring");

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, g = lane >> 5,
            r32 = lane & 31;
  const int wm = wave / WNN, wn = wave % WNN;
  const int64_t K = a.K, N = a.N;

  int e = 0, n_tile, m;
  int64_t row0;
  {
    const int x = (int)(blockIdx.x & 7u), j = (int)(blockIdx.x >> 3);
    if (a.offsets) {
      if (!w16_item<BM>(a.offsets, a.E, a.R, a.min_rows, a.max_rows, a.ntiles, x, j, e, n_tile, row0, m)) return;
    } else {  // the items of an n-tile are its units; 8 contiguous ranges of items, one per XCD
      const int64_t units = (a.R + BM - 1) / BM, total = units * a.ntiles, w = x * total / 8 + j;
      if (w >= (x + 1) * total / 8) return;
      n_tile = (int)(w / units);
      row0 = (w % units) * BM;
      m = (int)min((int64_t)BM, a.R - row0);
    }
  }
  const int64_t wrow = K / 2, srow = kNV ? K / 16 : K / 32, half = N / 2;
  const int nst = (int)(K / 64);

  const buf_rsrc ra = a.pair ? make_rsrc(a.a, (uint32_t)(a.a_rows * K * 2))
                             : make_rsrc(a.a + row0 * K, (uint32_t)((int64_t)m * K * 2));
  const buf_rsrc rb = make_rsrc(a.w + (int64_t)e * N * wrow, (uint32_t)(N * wrow));
  const buf_rsrc rbs = make_rsrc(a.ws + (int64_t)e * N * srow, (uint32_t)(N * srow));

  // the weight row that tile row r holds (N and beyond: reads as zero)
  auto b_row = [&](int r) -> int64_t {
    if (kSwiglu) return (r < BN / 2 ? 0 : half - BN / 2) + (int64_t)n_tile * (BN / 2) + r;
    return (int64_t)n_tile * BN + r;
  };
  uint32_t va[IA], vb[IB];
#pragma unroll
  for (int q = 0; q < IA; ++q) {
    const int chunk = (wave * IA + q) * 64 + lane, r = chunk >> 3;
    int64_t src = r;  // relative to row0; rows past m are past the resource
    if (a.pair) {
      src = a.a_rows;
      if (r < m) src = min((int64_t)((uint32_t)a.pair[row0 + r] / (uint32_t)a.topk), a.a_rows);
    }
    va[q] = (uint32_t)(src * K * 2 + 16 * ((chunk & 7) ^ swz_a16(r)));
  }
#pragma unroll
  for (int q = 0; q < IB; ++q) {
    const int chunk = (wave * IB + q) * 64 + lane, r = chunk >> 1;
    vb[q] = (uint32_t)(b_row(r) * wrow + 16 * ((chunk & 1) ^ swz_b16(r)));
  }
  const bool has_sc = wave < BN / 64;
  const uint32_t vs = (uint32_t)(b_row(64 * (has_sc ? wave : 0) + lane) * srow);

  auto issue = [&](W16Slot<BM, BN>& sl, int st) {
#pragma unroll
    for (int q = 0; q < IB; ++q) buf_dma16(rb, &sl.B[(wave * IB + q) * 1024], vb[q], (uint32_t)st * 32);
    if (has_sc) buf_dma4(rbs, &sl.Bs[wave * 256], vs, (uint32_t)(kNV ? 4 * st : 4 * (st >> 1)));
#pragma unroll
    for (int q = 0; q < IA; ++q) buf_dma16(ra, &sl.A[(wave * IA + q) * 1024], va[q], (uint32_t)st * 128);
  };

  v16f acc[2][FN];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int f = 0; f < FN; ++f) acc[i][f] = v16f{};
  int brow_l[FN], aoff[2], boff[FN];
#pragma unroll
  for (int f = 0; f < FN; ++f) {
    if (kSwiglu) brow_l[f] = (f < FN / 2 ? 0 : BN / 2) + FN * 16 * wn + 32 * (f % (FN > 1 ? FN / 2 : 1)) + r32;
    else brow_l[f] = 32 * (FN * wn + f) + r32;
    boff[f] = brow_l[f] * 32 + 16 * (g ^ swz_b16(brow_l[f]));
  }
#pragma unroll
  for (int f = 0; f < 2; ++f) {
    const int r = 64 * wm + 32 * f + r32;
    aoff[f] = r * 128 + 16 * ((4 * g) ^ swz_a16(r));
  }

  auto compute = [&](const W16Slot<BM, BN>& sl, int st) {
    v4i b[FN], av[2][4];
    uint32_t sd[FN];
#pragma unroll
    for (int f = 0; f < FN; ++f) {
      sd[f] = *reinterpret_cast<const uint32_t*>(&sl.Bs[4 * brow_l[f]]);
      b[f] = *reinterpret_cast<const v4i*>(&sl.B[boff[f]]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        int o = aoff[f];
        asm volatile("" : "+v"(o));
        av[f][j] = *reinterpret_cast<const v4i*>(&sl.A[o ^ (16 * j)]);
      }
    float sc[FN][2];
#pragma unroll
    for (int f = 0; f < FN; ++f) {
      if (kNV) {
        sc[f][0] = ue4m3_to_f32((sd[f] >> (16 * g)) & 0xFFu);
        sc[f][1] = ue4m3_to_f32((sd[f] >> (16 * g + 8)) & 0xFFu);
      } else {
        sc[f][0] = sc[f][1] = ue8m0_to_f32((sd[f] >> (8 * (2 * (st & 1) + g))) & 0xFFu);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int f = 0; f < FN; ++f) {
        const v8bf wv = kNV ? decode8_nv((uint32_t)b[f][j], sc[f][j >> 1]) : decode8((uint32_t)b[f][j], sc[f][0]);
#pragma unroll
        for (int fm = 0; fm < 2; ++fm) acc[fm][f] = mfma32x32x16(wv, __builtin_bit_cast(v8bf, av[fm][j]), acc[fm][f]);
      }
  };
  const bool active = 64 * wm < m;
  // stage st: wait for this wave's copies of st (those of st + 1 may stay in flight), meet
  // the others (their parts have landed too, and everyone is done with st - 1, whose slot
  // the copies of st + 2 overwrite), issue st + 2, compute st
  auto step = [&](auto I, int st) {
    constexpr int i = decltype(I)::value;
    if (st + 1 < nst) {
      if (has_sc) wait_vmcnt<IA + IB + 1>();
      else wait_vmcnt<IA + IB>();
    } else {
      wait_vmcnt<0>();
    }
    lds_barrier();
    if (st + 2 < nst) issue(ring[(i + 2) % kSlots], st + 2);
    __builtin_amdgcn_sched_barrier(0);
    if (active) compute(ring[i], st);
  };
  issue(ring[0], 0);
  if (nst > 1) issue(ring[1], 1);
  for (int st = 0; st < nst; st += kSlots) {
    step(std::integral_constant<int, 0>{}, st);
    if (st + 1 < nst) step(std::integral_constant<int, 1>{}, st + 1);
    if (st + 2 < nst) step(std::integral_constant<int, 2>{}, st + 2);
  }

  // adapters: for each segment with rows here, acc += low . lora_b^T over the rank, low
  // (scaled, fp32) split into two bf16 terms (16 significant bits: the adapter's share
  // keeps an error of 2^-17 of itself)
  if (kLora && active) {
    const int64_t rlo = row0 + 64 * wm, rhi = min(rlo + 64, row0 + m);
    for (int s = first_segment(a.seg_off, a.S, rlo); s < a.S; ++s) {
      const int64_t lo = a.seg_off[s], hi = a.seg_off[s + 1];
      if (lo >= rhi) break;
      const int l = a.seg_adapter[s];
      if (l < 0 || l >= a.L || hi <= rlo) continue;
      for (int k0 = 0; k0 < a.rank; k0 += 16) {
        const int k = k0 + 8 * g;
        v8bf xh[2], xl[2], bw[FN];
#pragma unroll
        for (int fm = 0; fm < 2; ++fm) {
          const int64_t t = rlo + 32 * fm + r32;
          const bool ok = t >= lo && t < hi && t < rhi && k < a.rank;
          float x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = 0.0f;
          if (ok) {
            for (int sl = 0; sl < a.nslice; ++sl) {
              const float4* p = reinterpret_cast<const float4*>(a.low + ((int64_t)sl * a.R + t) * a.rank + k);
              const float4 u = p[0], w = p[1];
              x[0] += u.x, x[1] += u.y, x[2] += u.z, x[3] += u.w;
              x[4] += w.x, x[5] += w.y, x[6] += w.z, x[7] += w.w;
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            xh[fm][i] = (__bf16)x[i];
            xl[fm][i] = (__bf16)(x[i] - (float)xh[fm][i]);
          }
        }
#pragma unroll
        for (int f = 0; f < FN; ++f) {
          const int64_t n = min((int64_t)n_tile * BN + brow_l[f], N - 1);
          v4i w = v4i{};
          if (k < a.rank) w = *reinterpret_cast<const v4i*>(a.lora_b + ((int64_t)l * N + n) * a.rank + k);
          bw[f] = __builtin_bit_cast(v8bf, w);
        }
#pragma unroll
        for (int f = 0; f < FN; ++f)
#pragma unroll
          for (int fm = 0; fm < 2; ++fm) {
            acc[fm][f] = mfma32x32x16(bw[f], xl[fm], acc[fm][f]);
            acc[fm][f] = mfma32x32x16(bw[f], xh[fm], acc[fm][f]);
          }
      }
    }
  }

  // epilogue: 32 rows x CP columns at a time through the wave's 8 KB of the ring (runs of
  // 4 columns in, 16-byte pieces of whole row segments out)
  lds_barrier();  // every wave is done with the ring
  if (!active) return;
  constexpr int ES = kOutBF16 ? 2 : 4, OF = kSwiglu ? FN / 2 : FN;
  constexpr int PF = OF * 32 * ES > 256 ? 256 / (32 * ES) : OF;  // fragments per pass
  constexpr int RB = PF * 32 * ES, NCH = RB / 16;
  static_assert(OF % PF == 0, "passes");
  uint8_t* const stg = reinterpret_cast<uint8_t*>(&ring[0]) + wave * 8192;
  const int64_t ocols = kSwiglu ? half : N;
  const int64_t col0 = ((int64_t)n_tile * BN >> (kSwiglu ? 1 : 0)) + OF * 32 * wn;
#pragma unroll
  for (int fm = 0; fm < 2; ++fm)
#pragma unroll
    for (int p = 0; p < OF / PF; ++p) {
#pragma unroll
      for (int f = 0; f < PF; ++f)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = acc[fm][p * PF + f][4 * j + i];
            if constexpr (kSwiglu) v[i] = silu_mul(x, acc[fm][p * PF + f + FN / 2][4 * j + i]);
            else v[i] = x;
          }
          if (kOutBF16) {
            const int c = (4 * f + j) ^ (r32 & (NCH - 1));
            *reinterpret_cast<uint2*>(stg + RB * r32 + 16 * c + 8 * g) =
                make_uint2(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]));
          } else {
            const int c = (8 * f + 2 * j + g) ^ (r32 & (NCH - 1));
            *reinterpret_cast<float4*>(stg + RB * r32 + 16 * c) = make_float4(v[0], v[1], v[2], v[3]);
          }
        }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
      for (int k = 0; k < NCH / 2; ++k) {
        const int idx = lane + 64 * k, rr = idx / NCH, c = idx % NCH;
        const v4i v = *reinterpret_cast<const v4i*>(stg + RB * rr + 16 * (c ^ (rr & (NCH - 1))));
        const int lrow = 64 * wm + 32 * fm + rr;
        const int64_t col = col0 + p * PF * 32 + c * (16 / ES);
        if (lrow < m && col < ocols)
          *reinterpret_cast<v4i*>(static_cast<uint8_t*>(a.out) + ((row0 + lrow) * ocols + col) * ES) = v;
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

template <int BM, int BN, int NW, bool kSwiglu, bool kLora>
void launch_shape(W16TileArgs a, bool nv, bool out_bf16, int64_t units, hipStream_t stream) {
  a.ntiles = (int)cdiv(a.N, BN);
  const dim3 grid((unsigned)(8 * cdiv(units * a.ntiles, 8))), block(NW * 64);
  if (nv) {
    if (out_bf16) w16_tile_kernel<BM, BN, NW, true, kSwiglu, true, kLora><<<grid, block, 0, stream>>>(a);
    else w16_tile_kernel<BM, BN, NW, true, kSwiglu, false, kLora><<<grid, block, 0, stream>>>(a);
  } else {
    if (out_bf16) w16_tile_kernel<BM, BN, NW, false, kSwiglu, true, kLora><<<grid, block, 0, stream>>>(a);
    else w16_tile_kernel<BM, BN, NW, false, kSwiglu, false, kLora><<<grid, block, 0, stream>>>(a);
  }
}

}  // namespace

void launch_w16_tile_grouped(const W16TileArgs& a, bool nv, bool swiglu, bool out_bf16, int bm, int64_t units,
                             hipStream_t stream) {
  if (bm == 256) {
    if (swiglu) launch_shape<256, 256, 8, true, false>(a, nv, out_bf16, units, stream);
    else launch_shape<256, 256, 8, false, false>(a, nv, out_bf16, units, stream);
  } else {
    if (swiglu) launch_shape<64, 256, 4, true, false>(a, nv, out_bf16, units, stream);
    else launch_shape<64, 256, 4, false, false>(a, nv, out_bf16, units, stream);
  }
}

void launch_w16_tile_lora(const W16TileArgs& a, bool nv, bool out_bf16, hipStream_t stream) {
  // 256 x 256 tiles once they fill the chip's 256 compute units; below that the small
  // tile's four times as many workgroups finish sooner
  if (cdiv(a.R, 256) * cdiv(a.N, 256) >= 256)
    launch_shape<256, 256, 8, false, true>(a, nv, out_bf16, cdiv(a.R, 256), stream);
  else launch_shape<64, 128, 4, false, true>(a, nv, out_bf16, cdiv(a.R, 64), stream);
}

}  // namespace mxf
