// Block norm (block_norm.hpp) of bf16 rows.
#include "block_norm.hpp"

namespace mxf {

int launch_block_norm(const BlockNormArgs& a, bool y_bf16, hipStream_t stream) {
  if (y_bf16) launch_k<true, 0>(a, stream);
  else launch_block_norm_f32(a, stream);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace mxf
