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
void launch_shape(W16TileArgs a, bool nv, bool out_bf16, int64_t units, hipStream_t stream) {
  a.ntiles = (int)cdiv(a.N, BN);
  const dim3 grid((unsigned)(8 * cdiv(units * a.ntiles, 8))), block(NW * 64);
  if (nv) {
    if (out_bf16) w16_tile_kernel<BM, BN, NW, NA, true, kSwiglu, true, kLora><<<grid, block, 0, stream>>>(a);
    else w16_tile_kernel<BM, BN, NW, NA, true, kSwiglu, false, kLora><<<grid, block, 0, stream>>>(a);
  } else {
    if (out_bf16) w16_tile_kernel<BM, BN, NW, NA, false, kSwiglu, true, kLora><<<grid, block, 0, stream>>>(a);
    else w16_tile_kernel<BM, BN, NW, NA, false, kSwiglu, false, kLora><<<grid, block, 0, stream>>>(a);
  }
}

}  // namespace

void launch_w16_tile_grouped(const W16TileArgs& a, bool nv, bool swiglu, bool out_bf16, W16Shape shape, int64_t units,
                             hipStream_t stream) {
  if (shape == W16Shape::k128x256) {
    if (swiglu) launch_shape<128, 256, 4, 2, true, false>(a, nv, out_bf16, units, stream);
    else launch_shape<128, 256, 4, 2, false, false>(a, nv, out_bf16, units, stream);
  } else if (shape == W16Shape::k64x128 && !swiglu) {
    launch_shape<64, 128, 4, 3, false, false>(a, nv, out_bf16, units, stream);
  } else {
    if (swiglu) launch_shape<64, 256, 4, 3, true, false>(a, nv, out_bf16, units, stream);
    else launch_shape<64, 256, 4, 3, false, false>(a, nv, out_bf16, units, stream);
  }
}

void launch_w16_tile_lora(const W16TileArgs& a, bool nv, bool out_bf16, hipStream_t stream) {
  // 128 x 256 tiles once there is about one for each of the 256 compute units (two fit one);
  // below that the small tile's four times as many workgroups finish sooner. Measured, us (64 x
  // 128 | 128 x 256): 4096 x 7168, 1500 rows 123 | 136, 2048 rows (256 tiles) 179 | 147, 8192 rows
  // 571 | 435; 2048 x 4096, 3000 rows (192 tiles) 75 | 83, 4096 rows 103 | 85. 256 x 256 tiles, one a
  // compute unit: 227 instead of 234 at 4096 x 4096 x 7168, where they fill the chip once, else slower.
  if (cdiv(a.R, 128) * cdiv(a.N, 256) >= 240) launch_shape<128, 256, 4, 2, false, true>(a, nv, out_bf16, cdiv(a.R, 128), stream);
  else launch_shape<64, 128, 4, 3, false, true>(a, nv, out_bf16, cdiv(a.R, 64), stream);
}

}  // namespace mxf
