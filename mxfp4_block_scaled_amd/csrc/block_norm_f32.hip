// Block norm (block_norm.hpp) of fp32 rows: a source of its own, so that the two compile side by side.
#include "block_norm.hpp"

namespace mxf {

void launch_block_norm_f32(const BlockNormArgs& a, hipStream_t stream) { launch_k<false, 0>(a, stream); }

}  // namespace mxf
