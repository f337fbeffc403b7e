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
  float* low;                 // kSplit: [slices][M][rank] fp32
  uint16_t *low_hi, *low_lo;  // else [M][rank] bf16 each, the sum's two terms
  int64_t M, K;
  int rank, L, S, zsplit;
};

// Workgroup (x, y, z): a block of 16 MF rows, K slice y, every zsplit-th segment of those
// rows from the z-th on. NW waves split the slice's K and meet in LDS in wave order. MF x RF
// fragments of 16 rows x 16 ranks on the 16x16x32 MFMA. Bound by the loads: a workgroup
// reads its rows' share of a once and the adapters of their segments; row blocks are dealt to
// the XCDs in contiguous ranges, so that an adapter is fetched into the L2 of the XCDs that
// use it only. A load instruction takes whole 128-byte lines of 8 rows (lanes that follow
// each other read what follows: the matrix lane layout, 16 rows in 16 neighbouring lanes,
// costs the address unit 64 accesses an instruction: 73 us instead of 37 for 4096 x 7168
// activations and rank 64);
// each fragment then passes through 2 KB of the wave's LDS into the lane layout.
template <int MF, int RF, int NW, bool kSplit>
__global__ void __launch_bounds__(NW * 64) lora_shrink_kernel(ShrinkArgs p) {
  constexpr int kArea = MF * RF * 1024 > 2048 ? MF * RF * 1024 : 2048;  // a fragment, then the partial sums
  __shared__ v4i part[NW][kArea / 16];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, g = lane >> 4, r16 = lane & 15, q = lane >> 3, j = lane & 7;
  const uint32_t nb = (uint32_t)((p.M + 16 * MF - 1) / (16 * MF));
  const int x = (int)(blockIdx.x & 7u);
  const uint32_t blk = w16_eighths(nb, x) + (blockIdx.x >> 3);
  if (blk >= w16_eighths(nb, x + 1)) return;
  const int64_t K = p.K, row0 = (int64_t)blk * (16 * MF), row1 = min(row0 + 16 * MF, p.M);
  const int nk = (int)(K / 64), ns = (int)gridDim.y * NW, me = (int)blockIdx.y * NW + wave;
  const int k0 = (int)((int64_t)me * nk / ns), k1 = (int)((int64_t)(me + 1) * nk / ns);
  const uint32_t krow = (uint32_t)(2 * K), voff = q * krow + 16 * j;
  const buf_rsrc ra = make_rsrc(p.a + row0 * K, (uint32_t)((row1 - row0) * K * 2));
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
  for (int s = first_segment(p.seg_off, p.S, row0) + (int)blockIdx.z; s < p.S; s += p.zsplit) {
    const int64_t s_lo = p.seg_off[s], s_hi = p.seg_off[s + 1];
    const int l = __builtin_amdgcn_readfirstlane(p.seg_adapter[s]);
    const int64_t lo = max(s_lo, row0), hi = min(s_hi, row1);
    if (s_lo >= row1) break;
    if (l < 0 || l >= p.L || hi <= lo) continue;
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
      const int64_t row = row0 + 16 * (i / (4 * RF)) + 4 * g + (i & 3);
      const int r = 16 * ((i >> 2) % RF) + r16;
      if (row < lo || row >= hi || r >= p.rank) continue;
      if (kSplit) {
        p.low[((int64_t)blockIdx.y * p.M + row) * p.rank + r] = t;
      } else {
        const __bf16 h = (__bf16)t, d = (__bf16)(t - (float)h);
        p.low_hi[row * p.rank + r] = __builtin_bit_cast(uint16_t, h);
        p.low_lo[row * p.rank + r] = __builtin_bit_cast(uint16_t, d);
      }
    }
    __syncthreads();  // the sums have been read: the areas are free for the next segment
  }
}

// One row of segments in 16: rows of a block, 32 only where blocks of 16 would be more than
// the compute units anyway and segments are long (an adapter is then read for twice the rows)
template <int RF>
void launch_shrink(const ShrinkArgs& s, int slices, hipStream_t stream) {
  const bool wide = s.M >= 32 * 256 && s.M >= 32 * (int64_t)s.S;
  const int64_t blocks = cdiv(s.M, wide ? 32 : 16);
  ShrinkArgs a = s;
  a.zsplit = (int)(cdiv(s.S, blocks) < 16 ? cdiv(s.S, blocks) : 16);
  const dim3 grid((unsigned)(8 * cdiv(blocks, 8)), (unsigned)slices, (unsigned)a.zsplit);
  constexpr int NW = RF == 8 ? 8 : 16;  // what fits the registers
  if (s.low) lora_shrink_kernel<1, RF, 8, true><<<grid, 512, 0, stream>>>(a);
  else if (wide) lora_shrink_kernel<2, RF, NW, false><<<grid, NW * 64, 0, stream>>>(a);
  else lora_shrink_kernel<1, RF, NW, false><<<grid, NW * 64, 0, stream>>>(a);
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
  const int s = first_segment(p.seg_off, p.S, t);
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
  // M <= 64: K slices of at least 512 (64 k for each of a workgroup's 8 waves), up to 8; more
  // rows: the waves of one workgroup take the whole K and low is final
  return M > 64 ? 1 : (int)(K / 512 < 8 ? K / 512 : 8);
}

int lora_base_slices(int64_t M, int64_t N, int64_t K) { return M <= 64 ? w4a16_ksplit(M, N, K) : 0; }

int launch_w16_lora(const W16LoraArgs& p, bool nv, bool out_bf16, hipStream_t stream) {
  const int ls = lora_shrink_slices(p.M, p.K);
  float* const base = p.workspace;
  float* const low = base + (int64_t)lora_base_slices(p.M, p.N, p.K) * p.M * p.N;
  uint16_t* const low_hi = reinterpret_cast<uint16_t*>(low);  // M > 64: two bf16 terms in fp32's place
  uint16_t* const low_lo = low_hi + p.M * p.rank;
  if (p.S > 0) {
    const ShrinkArgs s{p.a, p.lora_a, p.scaling, p.seg_off, p.seg_adapter, p.M > 64 ? nullptr : low, low_hi, low_lo,
                       p.M, p.K, p.rank, p.L, p.S, 1};
    if (p.rank <= 16) launch_shrink<1>(s, ls, stream);
    else if (p.rank <= 32) launch_shrink<2>(s, ls, stream);
    else if (p.rank <= 64) launch_shrink<4>(s, ls, stream);
    else launch_shrink<8>(s, ls, stream);
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
    a.low_hi = low_hi;
    a.low_lo = low_lo;
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
