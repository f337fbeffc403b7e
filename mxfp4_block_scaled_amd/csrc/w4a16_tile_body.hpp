// Tiled products of bf16 activations with FP4 weights: y = A . W_hat^T for many rows per
// weight matrix, either grouped by expert with ragged row ranges (moe_grouped_gemm_w4a16)
// or over one matrix with low-rank adapters beside it (fp4_gemm_w4a16_lora).
//
// A workgroup computes BM rows x BN weight rows with waves of 32 FM rows x 32 FN weight rows
// on the 32x32x16 bf16 MFMA (weights as the first operand, so a lane ends up with runs of
// 4 consecutive columns of one row). A stage is 64 k. Everything is copied HBM -> LDS
// directly: NA slots of BM x 128 bytes of activations, one stage each; two of BN x 64 bytes
// of codes, 128 k each; two of 16 scale bytes per weight row (512 k of MXFP4, 256 k of
// NVFP4). The wider pieces of codes and scales halve and quarter the number of cache lines
// that a copy asks for (12288 rows over 32 experts of 4096 x 7168: the copies alone 473 us
// with 32 bytes and one scale dword a stage, 357 so). The copies of stage st + NA - 1 go out
// while st is computed. The weights stay 4 bits wide up to the registers: a lane reads the 16
// bytes that hold 32 codes of its weight row and converts 8 of them (exactly: a code times
// its scale has at most 5 significant bits) in front of each MFMA.
//
// K order: inside a stage MFMA j takes, in lane group g (lane / 32), k = 32 g + 8 j +
// [0, 8), for both operands: a weight lane's 16 bytes are chunk 2 (st & 1) + g of its
// 64-byte code row, one 32-element block, and an activation lane reads chunk 4 g + j of its
// 128-byte stage row. Chunks are XOR-swizzled per row so that the 16 lanes of an LDS
// cycle hit different banks.
//
// Many rows are bound by the MFMA at the clock that the power allows: 32 experts x 4096 x
// 7168, 12288 rows, SwiGLU (0.72 TFLOP) 605-650 us by the card = 1.1-1.2 PFLOP/s, the MFMA busy 65 %
// of the time at 1.8 GHz; a plain bf16 product of the same size from the library 552 us. NVFP4 715-755 us,
// 50 %: its decoding multiplies each weight by the scale's mantissa first. There the 128 x
// 256 tile has two slots (73 KB: two workgroups a compute unit, whose stages interleave); 256
// x 256 and 128 x 512, one workgroup a compute unit, were slower (742 us). Without adapters a wave
// there takes all 128 rows, so that a weight is decoded once (2 experts of 4096 rows 426 -> 417 us
// against waves of 64 rows x 128), and half of the MFMAs where a unit has at most 64 rows. Few tiles are
// bound by the length of a stage, 0.36 us with 64 x 128 tiles: copy, barrier, decode and MFMA
// of one wave after each other. Three slots there; four or five take the room of a workgroup
// (256 rows x 4096 x 7168 in K slices 35 -> 38 us).
//
// Rows past a unit's end and weight rows past N read as zero through the range-checked
// buffer resources and are not stored.
#pragma once

#include "w4a16_tile.hpp"

namespace mxf {

// LDS: NA slots of one 64-k stage of activations, two of 128 k of weight codes, two of a
// scale group (16 scale bytes per weight row: 512 k of UE8M0 or 256 k of UE4M3)
template <int BM, int BN, int NA>
struct alignas(16) W16Ring {
  uint8_t A[NA][BM * 128];
  uint8_t B[2][BN * 64];
  uint8_t S[2][BN * 16];
};

__device__ __forceinline__ v16f mfma32x32x16(v8bf a, v8bf b, v16f c) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
#else
  (void)a;
  (void)b;
  return c;
#endif
}

// One workgroup's tile: BM x BN by NW waves, BM / (32 FM) of them over rows, the others over
// columns; x, j: its XCD and item. kSlices (one matrix, j = unit x ntiles + n-tile): only the
// K slice `slice` of a.kslices, whose sums go to slice `slice` of out, [kslices][R][N] fp32.
template <int BM, int BN, int NW, int NA, bool kNV, bool kSwiglu, bool kOutBF16, bool kLora, bool kSlices>
__device__ __forceinline__ void w16_tile(const W16TileArgs& a, W16Ring<BM, BN, NA>& ring, int x, int j, int slice) {
  constexpr int FM = BM == 128 && !kLora ? 4 : 2, WM = 32 * FM, WMN = BM / WM, WNN = NW / WMN, FN = BN / WNN / 32;
  constexpr int IA = BM * 8 / 64 / NW, IB = BN * 4 / 64 / NW;  // 16-byte copies per lane per 64 / 128 k
  constexpr int P = kNV ? 4 : 8;  // stages per scale group
  static_assert(IA >= 1 && IB >= 1 && BN / 64 <= NW && (!kSwiglu || FN % 2 == 0), "tile shape");
  static_assert(sizeof(ring) <= 160 * 1024 && sizeof(ring) >= NW * 8192, "the epilogue stages through the ring");

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, g = lane >> 5,
            r32 = lane & 31;
  const int wm = wave / WNN, wn = wave % WNN;
  const int64_t K = a.K, N = a.N;

  int e = 0, n_tile, m;
  int64_t row0;
  if constexpr (kSlices) {  // item j: the n-tiles of a unit of rows after each other
    n_tile = j % a.ntiles;
    row0 = (int64_t)(j / a.ntiles) * BM;
    m = (int)min((int64_t)BM, a.R - row0);
  } else {
    if (a.offsets) {
      if (!w16_item<BM>(a.offsets, a.E, a.R, a.min_rows, a.max_rows, a.ntiles, x, j, e, n_tile, row0, m)) return;
    } else {  // 8 contiguous ranges of items, one per XCD
      const uint32_t units = (uint32_t)((a.R + BM - 1) / BM), total = units * (uint32_t)a.ntiles;
      uint32_t w;
      if (!w16_range(total, x, j, w)) return;
      int unit;
      w16_place(w, units, (uint32_t)a.ntiles, n_tile, unit);
      row0 = (int64_t)unit * BM;
      m = (int)min((int64_t)BM, a.R - row0);
    }
  }
  const int64_t wrow = K / 2, srow = kNV ? K / 16 : K / 32, half = N / 2;
  // stages [st0, nst) of 64 k; st0 is even (slices are whole 128 k)
  const int st0 = kSlices ? 2 * (int)(w16_share((uint32_t)(K / 128), slice, a.kslices)) : 0;
  const int nst = kSlices ? 2 * (int)(w16_share((uint32_t)(K / 128), slice + 1, a.kslices)) : (int)(K / 64);

  const buf_rsrc ra = a.pair ? make_rsrc(a.a, (uint32_t)(a.a_rows * K * 2))
                             : make_rsrc(a.a + row0 * K, (uint32_t)((int64_t)m * K * 2));
  const buf_rsrc rb = make_rsrc(a.w + (int64_t)e * N * wrow, (uint32_t)(N * wrow));
  const buf_rsrc rbs = make_rsrc(a.ws + (int64_t)e * N * srow, (uint32_t)(N * srow));

  auto b_row = [&](int r) -> int64_t { return w16_weight_row(kSwiglu, BN, half, n_tile, r); };
  uint32_t va[IA], vb[IB];
#pragma unroll
  for (int q = 0; q < IB; ++q) {
    const int chunk = (wave * IB + q) * 64 + lane, r = chunk >> 2;
    vb[q] = (uint32_t)(b_row(r) * wrow + 16 * ((chunk & 3) ^ swz_b16(r)));
  }
  const bool has_sc = wave < BN / 64;
  const uint32_t vs = (uint32_t)(b_row(64 * (has_sc ? wave : 0) + lane) * srow);
  auto issue_a = [&](uint8_t* slot, int st) {
#pragma unroll
    for (int q = 0; q < IA; ++q) buf_dma16(ra, slot + (wave * IA + q) * 1024, va[q], (uint32_t)st * 128);
  };
  auto issue_b = [&](uint8_t* slot, int h) {
#pragma unroll
    for (int q = 0; q < IB; ++q) buf_dma16(rb, slot + (wave * IB + q) * 1024, vb[q], (uint32_t)h * 64);
  };
  auto issue_s = [&](int grp) {
    if (has_sc) buf_dma16(rbs, &ring.S[grp & 1][wave * 1024], vs, (uint32_t)grp * 16);
  };
  issue_s(st0 / P);
  issue_b(ring.B[0], st0 / 2);
  // rows past m are past the resource
#pragma unroll
  for (int q = 0; q < IA; ++q) {
    const int chunk = (wave * IA + q) * 64 + lane, r = chunk >> 3;
    int64_t src = r;  // relative to row0
    if (a.pair) {
      src = a.a_rows;
      if (r < m) src = min((int64_t)((uint32_t)a.pair[row0 + r] / (uint32_t)a.topk), a.a_rows);
    }
    va[q] = (uint32_t)(src * K * 2 + 16 * ((chunk & 7) ^ swz_a16(r)));
  }
#pragma unroll
  for (int i = 0; i < NA - 1; ++i)
    if (st0 + i < nst) issue_a(ring.A[i], st0 + i);

  // adapters: the first 64 segments of the wave's rows, on their way during the product
  const int64_t rlo = row0 + WM * wm, rhi = min(rlo + 64, row0 + m);
  int s0 = 0, seg_b0 = 0, seg_b1 = 0, seg_ad = -1;
  auto fetch_segments = [&]() {
    const int s = s0 + lane < a.S ? s0 + lane : -1;
    seg_b0 = a.seg_off[max(s, 0)];
    seg_b1 = a.seg_off[s + 1];
    seg_ad = a.seg_adapter[max(s, 0)];
  };
  if constexpr (kLora) {
    s0 = first_segment(a.seg_off, a.S, rlo);
    if (s0 < a.S) fetch_segments();
  }

  v16f acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int f = 0; f < FN; ++f) acc[i][f] = v16f{};
  int brow_l[FN], aoff[FM], boff[FN];
#pragma unroll
  for (int f = 0; f < FN; ++f) {
    if (kSwiglu) brow_l[f] = (f < FN / 2 ? 0 : BN / 2) + FN * 16 * wn + 32 * (f % (FN > 1 ? FN / 2 : 1)) + r32;
    else brow_l[f] = 32 * (FN * wn + f) + r32;
    boff[f] = brow_l[f] * 64 + 16 * (g ^ swz_b16(brow_l[f]));
  }
#pragma unroll
  for (int f = 0; f < FM; ++f) {
    const int r = WM * wm + 32 * f + r32;
    aoff[f] = r * 128 + 16 * ((4 * g) ^ swz_a16(r));
  }

  auto compute = [&](const uint8_t* As, const uint8_t* Bs, auto Odd, auto Rows, int st) {
    constexpr int nf = decltype(Rows)::value;  // fragments of 32 rows
    constexpr int odd = decltype(Odd)::value;  // stages of 128 k: blocks 0, 1 then 2, 3 of a row's codes
    const uint8_t* const Ss = &ring.S[(st / P) & 1][4 * (kNV ? st & 3 : (st & 7) >> 1)];
    v4i b[FN], av[nf][4];
    uint32_t sd[FN];
#pragma unroll
    for (int f = 0; f < FN; ++f) {
      int o = boff[f];
      asm volatile("" : "+v"(o));
      sd[f] = *reinterpret_cast<const uint32_t*>(Ss + 16 * brow_l[f]);
      b[f] = *reinterpret_cast<const v4i*>(Bs + (o ^ (32 * odd)));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int f = 0; f < nf; ++f) {
        int o = aoff[f];
        asm volatile("" : "+v"(o));
        av[f][j] = *reinterpret_cast<const v4i*>(As + (o ^ (16 * j)));
      }
    float sc[FN][2];
#pragma unroll
    for (int f = 0; f < FN; ++f) {
      if (kNV) {
        sc[f][0] = ue4m3_to_f32((sd[f] >> (16 * g)) & 0xFFu);
        sc[f][1] = ue4m3_to_f32((sd[f] >> (16 * g + 8)) & 0xFFu);
      } else {
        sc[f][0] = sc[f][1] = ue8m0_to_f32((sd[f] >> (8 * (2 * odd + g))) & 0xFFu);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int f = 0; f < FN; ++f) {
        const v8bf wv = kNV ? decode8_nv((uint32_t)b[f][j], sc[f][j >> 1]) : decode8((uint32_t)b[f][j], sc[f][0]);
#pragma unroll
        for (int fm = 0; fm < nf; ++fm) acc[fm][f] = mfma32x32x16(wv, __builtin_bit_cast(v8bf, av[fm][j]), acc[fm][f]);
      }
  };
  const bool active = WM * wm < m;
  // stage st: wait for the copies it needs, meet the other waves (their parts have landed
  // too, and everyone is done with stage st - 1), issue into what stage st - 1 freed, compute.
  // Order, slots and counts: w4a16_plan.hpp.
  auto next_s = [&](int st) { return w16_begins_scales(st, kSlices ? st0 : 0, P, nst); };
  auto step = [&](auto I, auto Rows, int st) {
    constexpr int i = decltype(I)::value;  // of the slots: st - st0 modulo whole turns
    if (st + 1 >= nst) wait_vmcnt<w16_in_flight(i, NA, IA, IB, true, false)>();
    else if (i % 2 == 1 && has_sc && next_s(st - 1)) wait_vmcnt<w16_in_flight(i, NA, IA, IB, false, true)>();
    else wait_vmcnt<w16_in_flight(i, NA, IA, IB, false, false)>();
    lds_barrier();
    if (w16_issues_codes(i, st, nst)) issue_b(ring.B[w16_code_slot(i + 2)], st / 2 + 1);
    if (i % 2 == 0 && next_s(st)) issue_s(st / P + 1);
    if (w16_issues_a(st, NA, nst)) issue_a(ring.A[w16_a_slot(i + NA - 1, NA)], st + NA - 1);
    __builtin_amdgcn_sched_barrier(0);
    if (active) compute(ring.A[w16_a_slot(i, NA)], ring.B[w16_code_slot(i)], std::integral_constant<int, i % 2>{}, Rows, st);
  };
  constexpr int U = w16_turn(NA);
  auto stages = [&](auto Rows) {
    for (int st = st0; st < nst; st += U)  // nst is even
      static_for<0, U / 2>([&](auto X_) {
        constexpr int X = 2 * decltype(X_)::value;
        if (st + X < nst) {
          step(std::integral_constant<int, X>{}, Rows, st + X);
          step(std::integral_constant<int, X + 1>{}, Rows, st + X + 1);
        }
      });
  };
  if (FM > 2 && m <= WM / 2) stages(std::integral_constant<int, FM / 2>{});  // half a unit of rows
  else stages(std::integral_constant<int, FM>{});

  lds_barrier();  // every wave is done with the ring
  if (!kLora && !active) return;
  uint8_t* const stg = reinterpret_cast<uint8_t*>(&ring) + wave * 8192;

  // adapters: for each segment with rows here, acc += low . lora_b^T over the rank, 32 ranks at a
  // time. A row has one adapter, so the tile's low is read once: its K slices are added in fp32, and
  // the sum t is split exactly into three bf16 terms t = x0 + x1 + x2, which the waves read from LDS
  // as operands. Each term is the leading 8 bits of what the ones before leave, so of t's sign and
  // never larger than t (rounded terms could overflow or differ in sign); an infinity is x0 alone.
  // 64 segments' bounds and adapters are read at once, and the operands of D further items are
  // loaded before the current ones are multiplied, so that many short segments cost their loads and
  // not their latency.
  if constexpr (kLora) {
    uint8_t* const terms = reinterpret_cast<uint8_t*>(&ring) + NW * 8192;  // [3][BM rows][32 ranks] bf16
    static_assert(sizeof(ring) >= NW * 8192 + 3 * BM * 64, "the terms stand behind the staging areas");
    auto stage_terms = [&](int rc) {
#pragma unroll 1
      for (int i = 0; i < BM * 4 / (NW * 64); ++i) {
        const int idx = (int)threadIdx.x + NW * 64 * i, r = idx >> 2, c = idx & 3;  // 8 ranks of a row
        float t[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (r < m && rc + 8 * c < a.rank) {
          const float* const p = a.low + (row0 + r) * a.rank + rc + 8 * c;
          float4 u[kMaxTileLowSlices][2];
#pragma unroll
          for (int sl = 0; sl < kMaxTileLowSlices; ++sl)
            if (sl < a.lslices) {
              u[sl][0] = *reinterpret_cast<const float4*>(p + sl * a.R * a.rank);
              u[sl][1] = *reinterpret_cast<const float4*>(p + sl * a.R * a.rank + 4);
            }
#pragma unroll
          for (int sl = 0; sl < kMaxTileLowSlices; ++sl)
            if (sl < a.lslices)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                t[4 * h] += u[sl][h].x, t[4 * h + 1] += u[sl][h].y, t[4 * h + 2] += u[sl][h].z, t[4 * h + 3] += u[sl][h].w;
        }
        uint32_t x[3][8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          x[0][k] = __float_as_uint(t[k]) & 0xFFFF0000u;
          const float d = __builtin_isinf(t[k]) ? 0.0f : t[k] - __uint_as_float(x[0][k]);
          x[1][k] = __float_as_uint(d) & 0xFFFF0000u;
          x[2][k] = __float_as_uint(d - __uint_as_float(x[1][k]));
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          v4i w;
#pragma unroll
          for (int h = 0; h < 4; ++h) w[h] = (int)(x[k][2 * h] >> 16 | (x[k][2 * h + 1] & 0xFFFF0000u));
          *reinterpret_cast<v4i*>(terms + k * BM * 64 + r * 64 + 16 * (c ^ swz_b16(r))) = w;
        }
      }
    };
    struct Ops {
      v4i b[FN];
      int first, end, k;  // the segment's rows (relative to rlo), the first of 16 ranks
    };
    uint32_t boff_l[FN];  // per-lane byte offsets; the item adds scalars only (rows past N of lora_b read as zero)
#pragma unroll
    for (int f = 0; f < FN; ++f) boff_l[f] = (uint32_t)((n_tile * BN + brow_l[f]) * a.rank + 8 * g) * 2;
    const uint32_t nrank = (uint32_t)N * (uint32_t)a.rank * 2;
    // An infinity or NaN of lora_b meets x0 only, which is 0 only where t is (or below 2^-133; the
    // other terms may be 0, and 0 times it is NaN); and it would reach the rows beside the segment:
    // those rows' sums wait in LDS meanwhile.
    auto not_finite = [&](const Ops& o) -> bool {
      uint32_t any = 0;  // exponents of all ones carry into the sign
#pragma unroll
      for (int f = 0; f < FN; ++f)
#pragma unroll
        for (int i = 0; i < 4; ++i) any |= ((uint32_t)o.b[f][i] & 0x7FFF7FFFu) + 0x00800080u;
      return __ballot((any & 0x80008000u) != 0) != 0;
    };
    float* const kept = reinterpret_cast<float*>(stg) + lane;
    constexpr int D = FN == 1 ? 4 : 2;  // items in flight
    const int s_first = s0;
    for (int rc = 0; rc < a.rank && a.S > 0; rc += 32) {
      const int rc_end = min(rc + 32, a.rank);
      int lo_l = 0, hi_l = 0, l_l = 0, k_next = rc_end;
      int lo = 0, hi = 0, l = 0;  // the segment of the item to load
      unsigned long long mask = 0;
      s0 = s_first;
      bool more = active && s0 < a.S;
      if (rc > 0 && more) fetch_segments();
      auto advance = [&]() -> bool {  // the next 16 ranks, else the next segment
        k_next += 16;
        if (k_next < rc_end) return true;
        while (mask == 0) {
          if (!more) return false;
          const bool in = s0 + lane < a.S;
          const int64_t b0 = seg_b0, b1 = seg_b1;
          l_l = seg_ad;
          lo_l = (int)(max(b0, rlo) - rlo);
          hi_l = (int)(min(b1, rhi) - rlo);
          mask = __ballot(in && b0 < rhi && b1 > rlo && hi_l > lo_l && l_l >= 0 && l_l < a.L);
          more = s0 + 64 < a.S && __ballot(in && b0 >= rhi) == 0;
          s0 += 64;
          if (more) fetch_segments();
        }
        const int i = __ffsll((long long)mask) - 1;
        mask &= mask - 1;
        lo = __builtin_amdgcn_readlane(lo_l, i);
        hi = __builtin_amdgcn_readlane(hi_l, i);
        l = __builtin_amdgcn_readlane(l_l, i);
        k_next = rc;
        return true;
      };
      auto load = [&](Ops& o) {
        const buf_rsrc rw = make_rsrc(a.lora_b + (int64_t)l * N * a.rank, nrank);
        o.first = lo;
        o.end = hi;
        o.k = k_next;
        const bool kin = k_next + 8 * g < a.rank;  // the last 8 of a rank that is no multiple of 16
#pragma unroll
        for (int f = 0; f < FN; ++f) {
          o.b[f] = v4i{};
          if (kin) o.b[f] = buf_load16(rw, boff_l[f], 2 * (uint32_t)k_next);
        }
      };
      Ops o[D];
      bool have[D];
#pragma unroll
      for (int d = 0; d < D; ++d) {
        have[d] = advance();
        if (have[d]) load(o[d]);
      }
      if (rc > 0) lds_barrier();  // the terms before have been read
      stage_terms(rc);
      lds_barrier();
      while (have[0]) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
          if (!have[d]) break;
          const bool odd = __builtin_expect(not_finite(o[d]), 0), apart = odd && (o[d].first > 0 || o[d].end < 64);
          v8bf x[2][3];
#pragma unroll
          for (int fm = 0; fm < 2; ++fm) {
            const int t = 32 * fm + r32, r = WM * wm + t;
            const uint8_t* const at = terms + r * 64 + 16 * ((((o[d].k - rc) >> 3) + g) ^ swz_b16(r));
            const bool in = t >= o[d].first && t < o[d].end;
#pragma unroll
            for (int k = 0; k < 3; ++k)
              x[fm][k] = __builtin_bit_cast(v8bf, in ? *reinterpret_cast<const v4i*>(at + k * BM * 64) : v4i{});
          }
#pragma unroll
          for (int f = 0; f < FN; ++f) {
            if (apart) {
#pragma unroll
              for (int i = 0; i < 32; ++i) kept[64 * i] = acc[i / 16][f][i % 16];
              asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            }
#pragma unroll
            for (int k = 2; k >= 0; --k) {
              v4i b = o[d].b[f];
              if (k > 0 && odd) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  if ((b[i] & 0x7F80) == 0x7F80) b[i] &= (int)0xFFFF0000u;
                  if ((b[i] & 0x7F800000) == 0x7F800000) b[i] &= 0xFFFF;
                }
              }
#pragma unroll
              for (int fm = 0; fm < 2; ++fm) acc[fm][f] = mfma32x32x16(__builtin_bit_cast(v8bf, b), x[fm][k], acc[fm][f]);
            }
            if (apart) {
#pragma unroll
              for (int fm = 0; fm < 2; ++fm) {
                const int t = 32 * fm + r32;
                if (t < o[d].first || t >= o[d].end) {
#pragma unroll
                  for (int i = 0; i < 16; ++i) acc[fm][f][i] = kept[64 * (16 * fm + i)];
                }
              }
              asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            }
          }
          have[d] = advance();
          if (have[d]) load(o[d]);
        }
      }
    }
    if (!active) return;
  }

  // epilogue: 32 rows x CP columns at a time through the wave's 8 KB of the ring (runs of
  // 4 columns in, 16-byte pieces of whole row segments out)
  constexpr int ES = kOutBF16 ? 2 : 4, OF = kSwiglu ? FN / 2 : FN;
  constexpr int PF = OF * 32 * ES > 256 ? 256 / (32 * ES) : OF;  // fragments per pass
  constexpr int RB = PF * 32 * ES, NCH = RB / 16;
  static_assert(OF % PF == 0, "passes");
  const int64_t ocols = kSwiglu ? half : N;
  uint8_t* const out = static_cast<uint8_t*>(a.out) + (kSlices ? (int64_t)slice * a.R * N * 4 : 0);
  const int64_t col0 = ((int64_t)n_tile * BN >> (kSwiglu ? 1 : 0)) + OF * 32 * wn;
#pragma unroll
  for (int fm = 0; fm < FM; ++fm)
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
        const int lrow = WM * wm + 32 * fm + rr;
        const int64_t col = col0 + p * PF * 32 + c * (16 / ES);
        if (lrow < m && col < ocols)
          *reinterpret_cast<v4i*>(out + ((row0 + lrow) * ocols + col) * ES) = v;
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

}  // namespace mxf
