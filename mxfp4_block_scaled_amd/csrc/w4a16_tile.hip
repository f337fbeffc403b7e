// Launches of the tiled FP4-weight x bf16-activation product (w4a16_tile_body.hpp).
#include "w4a16_tile_body.hpp"

namespace mxf {

namespace {

template <int BM, int BN, int NW, int NA, bool kNV, bool kSwiglu, bool kOutBF16, bool kLora>
__global__ void __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(2))) w16_tile_kernel(W16TileArgs a) {
  __shared__ W16Ring<BM, BN, NA> ring;
  w16_tile<BM, BN, NW, NA, kNV, kSwiglu, kOutBF16, kLora, false>(a, ring, (int)(blockIdx.x & 7u), (int)(blockIdx.x >> 3),
                                                                 0);
}

template <int BM, int BN, int NW, int NA, bool kSwiglu, bool kLora>
void launch_shape(W16TileArgs a, bool nv, bool out_bf16, const W16Launch& l, hipStream_t stream) {
  a.min_rows = l.min_rows;
  a.max_rows = l.max_rows;
  a.ntiles = (int)l.ntiles;
  const dim3 grid((unsigned)l.workgroups()), block(NW * 64);
  if (nv) {
    if (out_bf16) w16_tile_kernel<BM, BN, NW, NA, true, kSwiglu, true, kLora><<<grid, block, 0, stream>>>(a);
    else w16_tile_kernel<BM, BN, NW, NA, true, kSwiglu, false, kLora><<<grid, block, 0, stream>>>(a);
  } else {
    if (out_bf16) w16_tile_kernel<BM, BN, NW, NA, false, kSwiglu, true, kLora><<<grid, block, 0, stream>>>(a);
    else w16_tile_kernel<BM, BN, NW, NA, false, kSwiglu, false, kLora><<<grid, block, 0, stream>>>(a);
  }
}

}  // namespace

void launch_w16_tile_grouped(const W16TileArgs& a, bool nv, bool swiglu, bool out_bf16, const W16Launch& l,
                             hipStream_t stream) {
  if (l.bm == 128) {
    if (swiglu) launch_shape<128, 256, 4, 2, true, false>(a, nv, out_bf16, l, stream);
    else launch_shape<128, 256, 4, 2, false, false>(a, nv, out_bf16, l, stream);
  } else if (l.bn == 128) {
    launch_shape<64, 128, 4, 3, false, false>(a, nv, out_bf16, l, stream);
  } else {
    if (swiglu) launch_shape<64, 256, 4, 3, true, false>(a, nv, out_bf16, l, stream);
    else launch_shape<64, 256, 4, 3, false, false>(a, nv, out_bf16, l, stream);
  }
}

void launch_w16_tile_lora(const W16TileArgs& a, bool nv, bool out_bf16, const W16LoraPlan& p, hipStream_t stream) {
  const W16Launch l{p.bm, p.bn, 0, 0, cdiv(a.R, p.bm), cdiv(a.N, p.bn)};
  if (p.bm == 128) launch_shape<128, 256, 4, 2, false, true>(a, nv, out_bf16, l, stream);
  else launch_shape<64, 128, 4, 3, false, true>(a, nv, out_bf16, l, stream);
}

}  // namespace mxf
