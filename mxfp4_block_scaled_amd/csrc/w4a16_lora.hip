// Low-rank adapters of many requests beside one shared FP4 projection:
//   c[t] = a[t] . W_hat^T + scaling[l] * (a[t] . lora_a[l]^T) . lora_b[l]^T
// with l = seg_adapter[s] of the segment s that holds row t (negative: no adapter).
//   shrink:  low[t] = scaling[l] * a[t] . lora_a[l]^T in fp32
//   tiles enough to fill the chip: the shrink, then the tiled product (w4a16_tile_body.hpp),
//            which takes low . lora_b^T into its accumulators after the last stage, so c is
//            written once. A tile adds its rows' K slices of low and splits the fp32 sums once, into
//            three bf16 terms that give them back exactly (4096 x 4096 x 7168, rank 64, 227 us; as two
//            rounded terms slice by slice, 16 bits, 234; each wave splitting its operands itself 241).
//   fewer:   a launch in which some workgroups compute K slices of the projection's tiles and the
//            others shrink, then one pass that adds the slices and the fp32 expansion: at these
//            sizes a call costs its launches and the length of its K chain (256 requests of one
//            row at 4096 x 7168, rank 16: 77 us with whole-K tiles, whose last stage walks 64
//            segments, 35 us sliced).
// Measured: 4096 x 4096 x 7168, rank 64, 16 segments (0.25 TFLOP) 227-240 us by the card, of which the
// shrink 24-28, bound as the tiled product is (with no adapter in use 188-193); fp32 results 230, NVFP4
// 286; 64 requests of one row at 4096 x 7168, rank 16 (26 MB) 18 us (NVFP4 19), one row at rank 32 10
// us, two launches of which one lasts at least 3.4 us.
#include "w4a16_tile_body.hpp"

namespace mxf {

namespace {

struct ShrinkArgs {
  const uint16_t* a;
  const uint16_t* lora_a;
  const float* scaling;
  const int32_t* seg_off;
  const int32_t* seg_adapter;
  float* low;  // [slices][M][rank]
  int64_t M, K;
  int rank, L, S, zsplit, slices;
};

// A workgroup's shrink: row block blk of 16 MF rows, K slice `slice` of p.slices, every
// zsplit-th segment of those rows from the z-th on. NW waves split the slice's K and meet in
// LDS in wave order. MF x RF fragments of 16 rows x 16 ranks on the 16x16x32 MFMA. Bound by
// the loads: a workgroup reads its rows' share of a once and the adapters of their segments;
// the launches deal row blocks to the XCDs in contiguous ranges, so that an adapter is
// fetched into the L2 of the XCDs that use it only. A load instruction takes whole 128-byte
// lines of 8 rows, and each fragment then passes through 2 KB of the wave's LDS into the lane
// layout (loaded in that layout, 16 rows in 16 neighbouring lanes, it costs the address unit
// 64 accesses an instruction: 73 us instead of 37 for 4096 x 7168 activations and rank 64).
// With K slices, so that there is a workgroup for each compute unit, 24-28 us: 175 MB, as each 32
// rows read their adapters, at about 7 TB/s out of the caches.
template <int MF, int RF, int NW>
struct ShrinkLds {
  v4i part[NW][(MF * RF * 1024 > 2048 ? MF * RF * 1024 : 2048) / 16];  // per wave: a fragment, then its partial sums
};

template <int MF, int RF, int NW>
__device__ __forceinline__ void lora_shrink(const ShrinkArgs& p, ShrinkLds<MF, RF, NW>& lds, uint32_t blk, int slice, int z) {
  auto& part = lds.part;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, g = lane >> 4, r16 = lane & 15, q = lane >> 3, j = lane & 7;
  const int64_t K = p.K, row0 = (int64_t)blk * (16 * MF), row1 = min(row0 + 16 * MF, p.M);
  const int nk = (int)(K / 64), ns = p.slices * NW, me = slice * NW + wave;
  const int k0 = (int)((int64_t)me * nk / ns), k1 = (int)((int64_t)(me + 1) * nk / ns);
  const uint32_t krow = (uint32_t)(2 * K), voff = q * krow + 16 * j;
  uint8_t* const stg = reinterpret_cast<uint8_t*>(&part[wave][0]);
  // row r's 16-byte chunk c at chunk c ^ swz(r) of its 128 bytes: no bank conflicts either way
  const int wr0 = 128 * q + 16 * (j ^ q), wr1 = 128 * (8 + q) + 16 * (j ^ q ^ 1);
  const int rd0 = 128 * r16 + 16 * (g ^ (r16 & 7) ^ (r16 >> 3));
  auto to_lanes = [&](const v4i (&raw)[2], v8bf (&op)[2]) {  // op[t]: row r16, k = 32 t + 8 g + [0, 8)
    *reinterpret_cast<v4i*>(stg + wr0) = raw[0];
    *reinterpret_cast<v4i*>(stg + wr1) = raw[1];
    op[0] = __builtin_bit_cast(v8bf, *reinterpret_cast<const v4i*>(stg + rd0));
    op[1] = __builtin_bit_cast(v8bf, *reinterpret_cast<const v4i*>(stg + (rd0 ^ 64)));
  };
  for (int s = first_segment(p.seg_off, p.S, row0) + z; s < p.S; s += p.zsplit) {
    const int64_t s_lo = p.seg_off[s], s_hi = p.seg_off[s + 1];
    const int l = __builtin_amdgcn_readfirstlane(p.seg_adapter[s]);
    const int64_t lo = max(s_lo, row0), hi = min(s_hi, row1);
    if (s_lo >= row1) break;
    if (l < 0 || l >= p.L || hi <= lo) continue;
    // the fragments' rows start at the segment's first; past its last they read as zero
    const buf_rsrc ra = make_rsrc(p.a + lo * K, (uint32_t)((hi - lo) * K * 2));
    const buf_rsrc rb = make_rsrc(p.lora_a + (int64_t)l * p.rank * K, (uint32_t)(p.rank * krow));  // ranks past: zero
    v4f acc[MF][RF];
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
      for (int f = 0; f < RF; ++f) acc[m][f] = v4f{0.f, 0.f, 0.f, 0.f};
    constexpr int U = MF + RF <= 2 ? 4 : MF == 1 || RF <= 2 ? 2 : 1;  // 64-k steps per batch of loads
    for (int k = k0; k < k1; k += U) {
      v4i xr[U][MF][2], wr[U][RF][2];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t kk = 128u * (uint32_t)min(k + u, k1 - 1);  // a step past the share is read again and not used
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int m = 0; m < MF; ++m) xr[u][m][i] = buf_load16(ra, voff, (16 * m + 8 * i) * krow + kk);
#pragma unroll
          for (int f = 0; f < RF; ++f) wr[u][f][i] = buf_load16(rb, voff, (16 * f + 8 * i) * krow + kk);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (k + u >= k1) break;
        v8bf xo[MF][2];
#pragma unroll
        for (int m = 0; m < MF; ++m) to_lanes(xr[u][m], xo[m]);
#pragma unroll
        for (int f = 0; f < RF; ++f) {
          v8bf wo[2];
          to_lanes(wr[u][f], wo);
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int m = 0; m < MF; ++m)
              acc[m][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xo[m][t], wo[t], acc[m][f], 0, 0, 0);
        }
      }
    }
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
      for (int f = 0; f < RF; ++f)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          reinterpret_cast<float*>(stg)[((m * RF + f) * 4 + v) * 64 + lane] = acc[m][f][v];
    __syncthreads();
    const float scale = p.scaling[l];
    for (int i = wave; i < MF * RF * 4; i += NW) {
      float t = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) t += reinterpret_cast<const float*>(&part[w][0])[i * 64 + lane];
      t *= scale;
      const int64_t row = lo + 16 * (i / (4 * RF)) + 4 * g + (i & 3);
      const int r = 16 * ((i >> 2) % RF) + r16;
      if (row < hi && r < p.rank) p.low[((int64_t)slice * p.M + row) * p.rank + r] = t;
    }
    __syncthreads();  // the sums have been read: the areas are free for the next segment
  }
}

// Not sliced: grid (8 x row blocks of an XCD, K slices, segments' share)
template <int MF, int RF, int NW>
__global__ void __launch_bounds__(NW * 64) lora_shrink_kernel(ShrinkArgs p) {
  __shared__ ShrinkLds<MF, RF, NW> lds;
  const uint32_t nb = (uint32_t)((p.M + 16 * MF - 1) / (16 * MF));
  const int x = (int)(blockIdx.x & 7u);
  const uint32_t blk = w16_eighths(nb, x) + (blockIdx.x >> 3);
  if (blk < w16_eighths(nb, x + 1)) lora_shrink<MF, RF, NW>(p, lds, blk, (int)blockIdx.y, (int)blockIdx.z);
}

// Sliced: the first workgroups each take a tile of the projection over a K slice, the others
// shrink (their row block slowest)
template <int RF, bool kNV>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2))) lora_decode_kernel(ShrinkArgs p, W16TileArgs a) {
  __shared__ union Lds {
    ShrinkLds<1, RF, 4> s;
    W16Ring<64, 128, 3> ring;
  } lds;
  const int items = a.ntiles * (int)((a.R + 63) / 64), nbase = items * a.kslices, b = (int)blockIdx.x;
  if (b < nbase) {  // slice by slice; within a slice the tiles are spread over the XCDs
    w16_tile<64, 128, 4, 3, kNV, false, false, false, true>(a, lds.ring, 0, b % items, b / items);
  } else {
    const int per = p.slices * p.zsplit, i = (b - nbase) % per;
    lora_shrink<1, RF, 4>(p, lds.s, (uint32_t)((b - nbase) / per), i % p.slices, i / p.slices);
  }
}

template <int RF>
void launch_shrink(const ShrinkArgs& a, int rows, hipStream_t stream) {
  const dim3 grid((unsigned)(8 * cdiv(cdiv(a.M, rows), 8)), (unsigned)a.slices, (unsigned)a.zsplit);
  constexpr int NW = RF == 8 ? 8 : 16;  // what fits the registers
  if (rows == 32) lora_shrink_kernel<2, RF, 8><<<grid, 512, 0, stream>>>(a);
  else lora_shrink_kernel<1, RF, NW><<<grid, NW * 64, 0, stream>>>(a);
}

template <int RF>
void launch_decode(const ShrinkArgs& s, const W16TileArgs& a, bool nv, hipStream_t stream) {
  const int nshrink = s.S > 0 ? (int)cdiv(s.M, 16) * s.slices * s.zsplit : 0;
  const dim3 grid((unsigned)(nshrink + a.ntiles * cdiv(a.R, 64) * a.kslices));
  if (nv) lora_decode_kernel<RF, true><<<grid, 256, 0, stream>>>(s, a);
  else lora_decode_kernel<RF, false><<<grid, 256, 0, stream>>>(s, a);
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

// One row, 256 columns per workgroup of one wave: 4 columns per lane. Latency bound (a chain of
// segment lookup, low, sum over the rank): about 5 of the 18 us of 64 requests at 4096 x 7168.
// lora_b through LDS in whole lines instead of a lane's own rows: 18.6 us.
template <bool kOutBF16>
__global__ void __launch_bounds__(64) lora_finish_kernel(FinishArgs p) {
  __shared__ float low[128];
  const int64_t t = blockIdx.y;
  const int64_t n = (int64_t)blockIdx.x * 256 + 4 * threadIdx.x;
  // the slices' loads go out before the segment is looked up
  float4 u[kMaxBaseSlices];
#pragma unroll
  for (int i = 0; i < kMaxBaseSlices; ++i)
    if (i < p.bslices && n < p.N) u[i] = *reinterpret_cast<const float4*>(p.base + ((int64_t)i * p.M + t) * p.N + n);
  const int s = first_segment(p.seg_off, p.S, t);
  int l = -1;
  if (s < p.S && (int64_t)p.seg_off[s] <= t) l = p.seg_adapter[s];
  const bool has = l >= 0 && l < p.L;
  constexpr int PR = 16;  // ranks of lora_b loaded ahead, beside low
  v4i pb[4][PR / 8];
  const uint16_t* const brow = p.lora_b + ((int64_t)(has ? l : 0) * p.N + n) * p.rank;
  if (has && n < p.N) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int i = 0; i < PR / 8; ++i)
        if (8 * i < p.rank) pb[c][i] = *reinterpret_cast<const v4i*>(brow + c * p.rank + 8 * i);
  }
  if (has)
    for (int r = threadIdx.x; r < p.rank; r += 64) {
      float w[kMaxLowSlices], v = 0.0f;
#pragma unroll
      for (int i = 0; i < kMaxLowSlices; ++i)  // all on their way before the first is added
        w[i] = i < p.lslices ? p.low[((int64_t)i * p.M + t) * p.rank + r] : 0.0f;
#pragma unroll
      for (int i = 0; i < kMaxLowSlices; ++i) v += w[i];
      low[r] = v;
    }
  __syncthreads();
  if (n >= p.N) return;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kMaxBaseSlices; ++i)
    if (i < p.bslices) v[0] += u[i].x, v[1] += u[i].y, v[2] += u[i].z, v[3] += u[i].w;
  if (has) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float d = 0.0f;
      auto dot8 = [&](const v4i& w, int r) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          d = fmaf(low[r + 2 * i], __uint_as_float((uint32_t)w[i] << 16), d);
          d = fmaf(low[r + 2 * i + 1], __uint_as_float((uint32_t)w[i] & 0xFFFF0000u), d);
        }
      };
#pragma unroll
      for (int i = 0; i < PR / 8; ++i)
        if (8 * i < p.rank) dot8(pb[c][i], 8 * i);
      for (int r = PR; r < p.rank; r += 8) dot8(*reinterpret_cast<const v4i*>(brow + c * p.rank + r), r);
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

int launch_w16_lora(const W16LoraArgs& p, bool nv, bool out_bf16, hipStream_t stream) {
  const W16LoraPlan l = w16_lora_plan(p.M, p.N, p.K, p.rank, p.S);
  const int bs = l.base_slices, ls = l.low_slices;
  float* const base = p.workspace;
  float* const low = base + (int64_t)bs * p.M * p.N;
  const ShrinkArgs s{p.a, p.lora_a, p.scaling, p.seg_off, p.seg_adapter, low, p.M, p.K, p.rank, p.L, p.S, l.low_share,
                     ls};
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
  a.rank = p.rank;
  a.L = p.L;
  a.S = p.S;
  a.lslices = ls;
  a.kslices = bs;
  a.seg_off = p.seg_off;
  a.seg_adapter = p.seg_adapter;
  a.lora_b = p.lora_b;
  if (bs == 0) {
    if (p.S > 0) {
      if (p.rank <= 16) launch_shrink<1>(s, l.low_rows, stream);
      else if (p.rank <= 32) launch_shrink<2>(s, l.low_rows, stream);
      else if (p.rank <= 64) launch_shrink<4>(s, l.low_rows, stream);
      else launch_shrink<8>(s, l.low_rows, stream);
    }
    launch_w16_tile_lora(a, nv, out_bf16, l, stream);
  } else {
    a.out = base;
    a.ntiles = (int)cdiv(p.N, 128);
    if (p.rank <= 16) launch_decode<1>(s, a, nv, stream);
    else if (p.rank <= 32) launch_decode<2>(s, a, nv, stream);
    else if (p.rank <= 64) launch_decode<4>(s, a, nv, stream);
    else launch_decode<8>(s, a, nv, stream);
    FinishArgs f{base, low, p.lora_b, p.seg_off, p.seg_adapter, p.out, p.M, p.N, bs, ls, p.rank, p.L, p.S};
    const dim3 grid((unsigned)cdiv(p.N, 256), (unsigned)p.M);
    if (out_bf16) lora_finish_kernel<true><<<grid, 64, 0, stream>>>(f);
    else lora_finish_kernel<false><<<grid, 64, 0, stream>>>(f);
  }
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace mxf
