// Grouped products of bf16 activations with FP4 expert weights over ragged row ranges.
// Experts of at most 16 rows (decode, the tail of a skewed routing) stream their weights
// here, and so does all of a small call; the others run in the tiled kernel
// (w4a16_tile_body.hpp, launched from w4a16_tile.hip).
//
// The streaming kernel: a workgroup owns one expert and kSub runs, one after the other, of 64
// of its weight rows (SwiGLU: 32 gate rows and the 32 matching up rows); its 4 waves split K
// and meet in LDS in a fixed order. HBM bound: every weight byte is read once, as whole
// 128-byte lines with non-temporal loads, and passed through a per-wave LDS area into the
// lane layout of the 16x16x32 bf16 MFMA: lane (g, r16) holds the 32 codes of row r16, block
// 4 s + g of a 512-k super-step at step s, and instruction j takes their codes 8 j + [0, 8)
// against activations k = 128 s + 32 g + 8 j + [0, 8). Activations and scales pass through
// LDS too: loaded by the lane that needs them, 16 rows in 16 neighbouring lanes, they cost the
// address unit 64 accesses an instruction, and that was the bound (48 rows, which touch 44 or 45
// of 256 experts of 4096 x 7168, SwiGLU, 0.69 GB: 158 us with neither, 123 with the scales, 111 with
// both through LDS = 6.2 TB/s; NVFP4, 0.73 GB, 147 us = 5.0 TB/s, the vector unit busy 58 % of the time
// where it is 23 % with MXFP4). A launch that stays on the chip and walks the experts was slower (143 us), and so were a
// super-step's activations loaded one super-step ahead (115).
#include "w4a16_tile.hpp"

namespace mxf {

namespace {

constexpr int kStgStride = 1152;  // odd load instructions 128 B (mod 256) apart
constexpr int kStgBytes = 4 * kStgStride;

// A wave's LDS: one weight fragment on its way into the lane layout (afterwards the wave's
// partial sums), one step's activations, the super-step's scales
template <bool kNV>
struct alignas(16) W16StreamLds {
  uint8_t w[kStgBytes];
  uint8_t a[16 * 256];
  uint8_t s[64 * (kNV ? 32 : 16)];
};

template <bool kNV, bool kSwiglu, bool kOutBF16, int kSub>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(kNV ? 2 : 3))) w16_stream_kernel(W16TileArgs a) {
  __shared__ W16StreamLds<kNV> lds[4];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int e, n_run, m;
  int64_t row0;
  if (!w16_item<16>(a.offsets, a.E, a.R, a.min_rows, a.max_rows, a.ntiles, (int)(blockIdx.x & 7u),
                    (int)(blockIdx.x >> 3), e, n_run, row0, m))
    return;
  for (int sub = 0; sub < kSub; ++sub) {
    const int n_tile = n_run * kSub + sub;
    int lane = threadIdx.x & 63;
    if (kSub > 1) {
      if ((int64_t)n_tile * 64 >= a.N) return;
      if (sub > 0) __syncthreads();  // the sums before have been read
      asm volatile("" : "+v"(lane));  // formed anew: no registers are kept over a run
    }
    const int g = lane >> 4, r16 = lane & 15;
    const int64_t K = a.K, N = a.N, half = N / 2, wrow = K / 2, srow = kNV ? K / 16 : K / 32;

    // four 16-row weight fragments; those past the end read the first one again (not stored)
    const int64_t i0 = (int64_t)n_tile * (kSwiglu ? 32 : 64);
    const int64_t ocols = kSwiglu ? half : N;
    auto frag_row = [&](int f) -> int64_t {
      const int64_t c = i0 + 16 * (kSwiglu ? f & 1 : f);
      return (c < ocols ? c : i0) + (kSwiglu && f >= 2 ? half : 0);
    };
    const buf_rsrc wr = make_rsrc(a.w + (int64_t)e * N * wrow, (uint32_t)(N * wrow));
    const buf_rsrc sr = make_rsrc(a.ws + (int64_t)e * N * srow, (uint32_t)(N * srow));
    const int q = lane >> 3, rot = ((lane & 7) + q) & 7;
    const uint32_t wvoff = (uint32_t)(q * wrow + 16 * rot);
    const uint32_t svoff = (uint32_t)(frag_row(g) * srow + r16 * srow);  // lane 16 f + r: row r of fragment f
    uint8_t *const stg = lds[wave].w, *const sta = lds[wave].a, *const sts = lds[wave].s;
    int rd[4];
#pragma unroll
    for (int s = 0; s < 4; ++s)
      rd[s] = (2 * (s >> 1) + (r16 >> 3)) * kStgStride + 128 * (r16 & 7) + 16 * ((4 * s + g - (r16 & 7)) & 7);
    // activations: a load covers 4 rows x 256 bytes (a step's 128 k); rows past m read as zero
    const buf_rsrc ar = a.pair ? make_rsrc(a.a, (uint32_t)(a.a_rows * K * 2))
                               : make_rsrc(a.a + row0 * K, (uint32_t)((int64_t)m * K * 2));
    const bool few = m <= 4;
    int pr[4];  // looked at after the first weight loads have gone out
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * i + g;
      pr[i] = a.pair && r < m ? a.pair[row0 + r] : -1;
    }
    const int arow = min(r16, m - 1);

    v4f acc[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) acc[f] = v4f{0.f, 0.f, 0.f, 0.f};
    const int nss = (int)cdiv(K, 512);
    const int ss_begin = wave * nss / 4, ss_end = (wave + 1) * nss / 4;
    constexpr int SH = kNV ? 2 : 1;  // 16-byte pieces of a row's scale bytes per super-step
    for (int ss = ss_begin; ss < ss_end; ++ss) {
      const int steps = min(4, (int)(K / 128) - 4 * ss);  // 128-k steps of the super-step
      // every weight line and scale of the super-step is in flight before any wait (scale
      // bytes past the last row's end read as zero, dword by dword: a step past K is not run)
      v4i raw[4][4], sd[SH], ax[4];
#pragma unroll
      for (int h = 0; h < SH; ++h) sd[h] = buf_load16(sr, svoff, (uint32_t)(ss * 16 * SH + 16 * h));
#pragma unroll
      for (int f = 0; f < 4; ++f)
#pragma unroll
        for (int s = 0; s < 4; ++s)
          raw[f][s] = buf_load16_nt(wr, wvoff + 128 * (s >> 1),
                                    (uint32_t)((frag_row(f) + 8 * (s & 1)) * wrow + ss * 256));
      __builtin_amdgcn_sched_barrier(0);
      auto avoff = [&](int i) -> uint32_t {
        const uint32_t src = a.pair ? min((uint32_t)pr[i] / (uint32_t)a.topk, (uint32_t)a.a_rows) : (uint32_t)(4 * i + g);
        return src * (uint32_t)(2 * K) + 16 * r16;
      };
      // at most 4 rows: a load per step, all of them now; else the rows of step 0
      if (few) {
#pragma unroll
        for (int s = 0; s < 4; ++s) ax[s] = buf_load16(ar, avoff(0), (uint32_t)(ss * 1024 + 256 * w16_held_step(s, steps)));
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) ax[i] = buf_load16(ar, avoff(i), (uint32_t)(ss * 1024));
      }
      __builtin_amdgcn_sched_barrier(0);
      // a wave's LDS operations run in order: one area serves the fragments in turn
#pragma unroll
      for (int h = 0; h < SH; ++h) *reinterpret_cast<v4i*>(sts + 16 * (SH * lane + h)) = sd[h];
      v4i b[4][4];
#pragma unroll
      for (int f = 0; f < 4; ++f) {
#pragma unroll
        for (int s = 0; s < 4; ++s) *reinterpret_cast<v4i*>(stg + s * kStgStride + 16 * lane) = raw[f][s];
#pragma unroll
        for (int s = 0; s < 4; ++s) b[f][s] = *reinterpret_cast<const v4i*>(stg + rd[s]);
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (s >= steps) break;
        // row r's 16-byte chunk c sits at chunk c ^ r of its 256 bytes: no bank conflicts
        if (few) {
          *reinterpret_cast<v4i*>(sta + 256 * g + 16 * (r16 ^ g)) = ax[s];
        } else {
          if (s > 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) ax[i] = buf_load16(ar, avoff(i), (uint32_t)(ss * 1024 + 256 * s));
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<v4i*>(sta + 256 * (4 * i + g) + 16 * (r16 ^ (4 * i + g))) = ax[i];
        }
        v4i av[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) av[j] = *reinterpret_cast<const v4i*>(sta + 256 * arow + 16 * ((4 * g + j) ^ arow));
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          float sc[2];
          const uint32_t dw = *reinterpret_cast<const uint32_t*>(sts + 16 * SH * (16 * f + r16) + 4 * SH * s + (kNV ? 4 * (g >> 1) : 0));
          if constexpr (kNV) {
            sc[0] = ue4m3_to_f32((dw >> (16 * (g & 1))) & 0xFFu);
            sc[1] = ue4m3_to_f32((dw >> (16 * (g & 1) + 8)) & 0xFFu);
          } else {
            sc[0] = sc[1] = ue8m0_to_f32((dw >> (8 * g)) & 0xFFu);
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
      for (int v = 0; v < 4; ++v) reinterpret_cast<float*>(stg)[(4 * v + f) * 64 + lane] = acc[f][v];
    __syncthreads();
    constexpr int kW = sizeof(W16StreamLds<kNV>) / 4;
    float tot[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const float* r = reinterpret_cast<const float*>(lds[0].w) + (4 * wave + f) * 64 + lane;
      tot[f] = ((r[0] + r[kW]) + r[2 * kW]) + r[3 * kW];
    }
    const int lr = 4 * g + wave;
    if (lr < m) {
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
  }
}

template <bool kNV, bool kSwiglu, int kSub>
void launch_stream_t(const W16TileArgs& a, bool out_bf16, dim3 grid, hipStream_t stream) {
  if (out_bf16) w16_stream_kernel<kNV, kSwiglu, true, kSub><<<grid, 256, 0, stream>>>(a);
  else w16_stream_kernel<kNV, kSwiglu, false, kSub><<<grid, 256, 0, stream>>>(a);
}

template <bool kNV, int kSub>
void launch_stream_s(const W16TileArgs& a, bool swiglu, bool out_bf16, dim3 grid, hipStream_t stream) {
  if (swiglu) launch_stream_t<kNV, true, kSub>(a, out_bf16, grid, stream);
  else launch_stream_t<kNV, false, kSub>(a, out_bf16, grid, stream);
}

void launch_stream(W16TileArgs a, bool nv, bool swiglu, bool out_bf16, const W16Launch& l, hipStream_t stream) {
  a.min_rows = l.min_rows;
  a.max_rows = l.max_rows;
  a.ntiles = (int)l.ntiles;
  const dim3 grid((unsigned)l.workgroups());
  if (nv) launch_stream_s<true, 1>(a, swiglu, out_bf16, grid, stream);
  else if (l.bn == 256) launch_stream_s<false, 4>(a, swiglu, out_bf16, grid, stream);
  else launch_stream_s<false, 1>(a, swiglu, out_bf16, grid, stream);
}

}  // namespace

int launch_w16_grouped(const W16TileArgs& a, bool nv, bool swiglu, bool out_bf16, hipStream_t stream) {
  W16Launch l[3];
  const int n = w16_grouped_plan(a.R, a.E, a.N, a.K, nv, swiglu, l);
  for (int i = 0; i < n; ++i) {
    if (l[i].bm == 16) launch_stream(a, nv, swiglu, out_bf16, l[i], stream);
    else launch_w16_tile_grouped(a, nv, swiglu, out_bf16, l[i], stream);
  }
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace mxf
