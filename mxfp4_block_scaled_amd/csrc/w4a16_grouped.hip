// Grouped products of bf16 activations with FP4 expert weights over ragged row ranges.
// Experts of at most 16 rows (decode, the tail of a skewed routing) stream their weights
// here; the others run in the tiled kernel (w4a16_tile.hip).
//
// The streaming kernel: a workgroup owns one expert and 64 of its weight rows (SwiGLU: 32
// gate rows and the 32 matching up rows), its 4 waves split K and meet in LDS in a fixed
// order. HBM bound: every weight byte is read once, as whole 128-byte lines with
// non-temporal loads, and passed through a per-wave LDS area into the lane layout of the
// 16x16x32 bf16 MFMA: lane (g, r16) holds the 32 codes of row r16, block 4 s + g of a
// 512-k super-step at step s, and instruction j takes their codes 8 j + [0, 8) against
// activations k = 128 s + 32 g + 8 j + [0, 8).
#include "w4a16_tile.hpp"

namespace mxf {

namespace {

constexpr int kStgStride = 1152;  // odd load instructions 128 B (mod 256) apart
constexpr int kStgBytes = 4 * kStgStride;

template <bool kNV, bool kSwiglu, bool kOutBF16>
__global__ void __launch_bounds__(256) w16_stream_kernel(W16TileArgs a) {
  __shared__ v4i lds[4][4 * kStgBytes / 16];  // >= 4 KB per wave for the partial sums
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, g = lane >> 4, r16 = lane & 15;
  int e, n_tile, m;
  int64_t row0;
  if (!w16_item<0>(a.offsets, a.E, a.R, a.min_rows, a.max_rows, a.ntiles, (int)(blockIdx.x & 7u),
                   (int)(blockIdx.x >> 3), e, n_tile, row0, m))
    return;
  const int64_t K = a.K, N = a.N, half = N / 2, wrow = K / 2, srow = kNV ? K / 16 : K / 32;

  // four 16-row weight fragments; those past the end read the first one again (not stored)
  const int64_t i0 = (int64_t)n_tile * (kSwiglu ? 32 : 64);
  const int64_t ocols = kSwiglu ? half : N;
  int64_t frow[4];
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    const int64_t c = i0 + 16 * (kSwiglu ? f & 1 : f);
    frow[f] = (c < ocols ? c : i0) + (kSwiglu && f >= 2 ? half : 0);
  }
  buf_rsrc wr[4], sr[4];
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    wr[f] = make_rsrc(a.w + ((int64_t)e * N + frow[f]) * wrow, (uint32_t)(16 * wrow));
    sr[f] = make_rsrc(a.ws + ((int64_t)e * N + frow[f]) * srow, (uint32_t)(16 * srow));
  }
  const int q = lane >> 3, rot = ((lane & 7) + q) & 7;
  const uint32_t wvoff = (uint32_t)(q * wrow + 16 * rot);
  const uint32_t svoff = (uint32_t)(r16 * srow);
  uint8_t* const stg = reinterpret_cast<uint8_t*>(&lds[wave][0]);
  int rd[4];
#pragma unroll
  for (int s = 0; s < 4; ++s)
    rd[s] = (2 * (s >> 1) + (r16 >> 3)) * kStgStride + 128 * (r16 & 7) + 16 * ((4 * s + g - (r16 & 7)) & 7);
  // rows past m repeat row m - 1 (not stored)
  int64_t src = row0 + min(r16, m - 1);
  if (a.pair) src = min((int64_t)((uint32_t)a.pair[src] / (uint32_t)a.topk), a.a_rows - 1);
  const uint16_t* const ap = a.a + src * K + 32 * g;

  v4f acc[4];
#pragma unroll
  for (int f = 0; f < 4; ++f) acc[f] = v4f{0.f, 0.f, 0.f, 0.f};
  const int nss = (int)cdiv(K, 512);
  const int ss_begin = wave * nss / 4, ss_end = (wave + 1) * nss / 4;
  for (int ss = ss_begin; ss < ss_end; ++ss) {
    const int steps = min(4, (int)(K / 128) - 4 * ss);  // 128-k steps of the super-step
    v4i raw[4][4];
    uint32_t sd[4][kNV ? 8 : 4];  // the row's scale bytes of the super-step, a dword per step (MXFP4) or half step
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      constexpr int SD = kNV ? 8 : 4;
#pragma unroll
      for (int h = 0; h < SD; ++h) sd[f][h] = (uint32_t)buf_load4(sr[f], svoff, (uint32_t)(ss * 4 * SD + 4 * h));
#pragma unroll
      for (int s = 0; s < 4; ++s)
        raw[f][s] = buf_load16_nt(wr[f], wvoff + 128 * (s >> 1), (uint32_t)(8 * (s & 1) * wrow + ss * 256));
    }
    __builtin_amdgcn_sched_barrier(0);
    v4i b[4][4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      uint8_t* const area = stg + f * kStgBytes;
#pragma unroll
      for (int s = 0; s < 4; ++s) *reinterpret_cast<v4i*>(area + s * kStgStride + 16 * lane) = raw[f][s];
#pragma unroll
      for (int s = 0; s < 4; ++s) b[f][s] = *reinterpret_cast<const v4i*>(area + rd[s]);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s >= steps) break;
      v4i av[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) av[j] = *reinterpret_cast<const v4i*>(ap + (int64_t)ss * 512 + 128 * s + 8 * j);
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        float sc[2];
        if constexpr (kNV) {
          const uint32_t dw = sd[f][2 * s + (g >> 1)] >> (16 * (g & 1));
          sc[0] = ue4m3_to_f32(dw & 0xFFu);
          sc[1] = ue4m3_to_f32((dw >> 8) & 0xFFu);
        } else {
          sc[0] = sc[1] = ue8m0_to_f32((sd[f][s] >> (8 * g)) & 0xFFu);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const v8bf wv = kNV ? decode8_nv((uint32_t)b[f][s][j], sc[j >> 1]) : decode8((uint32_t)b[f][s][j], sc[0]);
          acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, av[j]), wv, acc[f], 0, 0, 0);
        }
      }
    }
  }
  // the waves' K shares in wave order; wave w finishes rows 4 g + w
  __syncthreads();
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int v = 0; v < 4; ++v) reinterpret_cast<float*>(&lds[wave][0])[(4 * v + f) * 64 + lane] = acc[f][v];
  __syncthreads();
  constexpr int kW = 4 * kStgBytes / 4;
  float tot[4];
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    const float* r = reinterpret_cast<const float*>(&lds[0][0]) + (4 * wave + f) * 64 + lane;
    tot[f] = ((r[0] + r[kW]) + r[2 * kW]) + r[3 * kW];
  }
  const int lr = 4 * g + wave;
  if (lr >= m) return;
#pragma unroll
  for (int f = 0; f < (kSwiglu ? 2 : 4); ++f) {
    float v;
    if constexpr (kSwiglu) v = silu_mul(tot[f], tot[f + 2]);
    else v = tot[f];
    const int64_t c = i0 + 16 * f;
    if (c >= ocols) continue;
    const int64_t at = (row0 + lr) * ocols + c + r16;
    if (kOutBF16) static_cast<uint16_t*>(a.out)[at] = (uint16_t)bf16x2_bits(v, 0.0f);
    else static_cast<float*>(a.out)[at] = v;
  }
}

template <bool kNV, bool kSwiglu>
void launch_stream_t(const W16TileArgs& a, bool out_bf16, dim3 grid, hipStream_t stream) {
  if (out_bf16) w16_stream_kernel<kNV, kSwiglu, true><<<grid, 256, 0, stream>>>(a);
  else w16_stream_kernel<kNV, kSwiglu, false><<<grid, 256, 0, stream>>>(a);
}

void launch_stream(W16TileArgs a, bool nv, bool swiglu, bool out_bf16, int64_t units, hipStream_t stream) {
  a.ntiles = (int)cdiv(a.N, 64);
  const dim3 grid((unsigned)(8 * cdiv(units * a.ntiles, 8)));
  if (nv && swiglu) launch_stream_t<true, true>(a, out_bf16, grid, stream);
  else if (nv) launch_stream_t<true, false>(a, out_bf16, grid, stream);
  else if (swiglu) launch_stream_t<false, true>(a, out_bf16, grid, stream);
  else launch_stream_t<false, false>(a, out_bf16, grid, stream);
}

// units that experts of lo < rows <= hi can make of R rows in all
int64_t most_units(int64_t R, int E, int64_t lo, int bm) {
  const int64_t experts = R / (lo + 1) < E ? R / (lo + 1) : E;
  return bm == 0 ? experts : experts + R / bm;
}

}  // namespace

int launch_w16_grouped(W16TileArgs a, bool nv, bool swiglu, bool out_bf16, hipStream_t stream) {
  constexpr int kAll = 0x7FFFFFFF;
  const int64_t R = a.R;
  a.min_rows = 0;
  a.max_rows = 16;
  launch_stream(a, nv, swiglu, out_bf16, most_units(R, a.E, 0, 0), stream);
  if (R > 16) {
    a.min_rows = 16;
    a.max_rows = 64;
    launch_w16_tile_grouped(a, nv, swiglu, out_bf16, 64, most_units(R, a.E, 16, 0), stream);
  }
  if (R > 64) {
    a.min_rows = 64;
    a.max_rows = kAll;
    launch_w16_tile_grouped(a, nv, swiglu, out_bf16, 256, most_units(R, a.E, 64, 256), stream);
  }
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace mxf
