// extern "C" entry points of the operators of training: the router's losses and gradient, the
// combine's backward pass, 4-bit quantisation both ways. Validation as in abi.cpp.
#include "abi_checks.hpp"
#include "fp4_pair_plan.hpp"
#include "launch.hpp"
#include "w4a16_plan.hpp"

using namespace mxf_abi;

namespace {
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int route_sizes(int64_t T, int32_t E, int32_t topk, int32_t S) {
  if (T < 0 || E < 1 || topk < 1 || topk > 8 || topk > E || S < 1) return MXF_ERR_SHAPE;
  if (E > 1024 || T > kMaxRows || T * (int64_t)topk > kMaxRows) return MXF_ERR_UNSUPPORTED;
  // one wave per token; pairs of a sequence and 64 experts counted in 32 bits
  if (mxf::cdiv(T, 4) * 256 > mxf::kMaxThreads || S * mxf::cdiv(E, 64) >= (int64_t(1) << 23)) return MXF_ERR_UNSUPPORTED;
  return MXF_OK;
}
}  // namespace

extern "C" {

size_t moe_balance_loss_workspace_bytes(int64_t T, int32_t E, int32_t S) {
  if (T < 0 || E < 1 || S < 1) return 0;
  return round_up(mxf::route_loss_workspace(T, E, S), 256);
}

int moe_balance_loss(const void* logits, int logits_dtype, const int32_t* topk_ids, const uint8_t* token_mask,
                     const int32_t* seg_offsets, int32_t S, int64_t T, int32_t E, int32_t topk, int32_t* counts,
                     int32_t* tokens, float* prob_mean, float* lse, float* losses, void* workspace,
                     size_t workspace_bytes, mxf_stream stream) {
  if (!valid_dtype(logits_dtype)) return MXF_ERR_FORMAT;
  if (const int rc = route_sizes(T, E, topk, S)) return rc;
  if (!seg_offsets && S != 1) return MXF_ERR_NULL;
  if (!counts || !tokens || !prob_mean || !losses || (T > 0 && (!logits || !topk_ids || !lse))) return MXF_ERR_NULL;
  const void* ptrs[] = {logits, topk_ids, seg_offsets, counts, tokens, prob_mean, lse, losses, workspace};
  if (!all_aligned16(ptrs)) return MXF_ERR_ALIGN;
  const size_t need = moe_balance_loss_workspace_bytes(T, E, S);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MXF_ERR_WORKSPACE;
  mxf::RouteLossArgs a{};
  a.logits = logits;
  a.topk_ids = topk_ids;
  a.token_mask = token_mask;
  a.seg_offsets = seg_offsets;
  a.T = T;
  a.E = E;
  a.topk = topk;
  a.S = S;
  a.counts = counts;
  a.tokens = tokens;
  a.prob_mean = prob_mean;
  a.lse = lse;
  a.losses = losses;
  a.workspace = workspace;
  return mxf::launch_route_loss(a, logits_dtype == MXF_BF16, as_stream(stream)) ? MXF_ERR_LAUNCH : MXF_OK;
}

int moe_route_backward(const void* logits, int logits_dtype, const int32_t* topk_ids, const float* gates,
                       const float* dgates, const float* dlosses, const float* lse, const int32_t* counts,
                       const int32_t* tokens, const int32_t* seg_offsets, int32_t S, int64_t T, int32_t E, int32_t topk,
                       void* dlogits, mxf_stream stream) {
  if (!valid_dtype(logits_dtype)) return MXF_ERR_FORMAT;
  if (const int rc = route_sizes(T, E, topk, S)) return rc;
  if (T == 0) return MXF_OK;
  if (!dlogits || (!dgates && !dlosses)) return MXF_ERR_NULL;
  if (dgates && (!gates || !topk_ids)) return MXF_ERR_NULL;
  if (dlosses && (!logits || !lse || !counts || !tokens || (!seg_offsets && S != 1))) return MXF_ERR_NULL;
  const void* ptrs[] = {logits, topk_ids, gates, dgates, lse, counts, tokens, seg_offsets, dlogits};
  if (!all_aligned16(ptrs) || !aligned4(dlosses)) return MXF_ERR_ALIGN;
  mxf::RouteLossArgs a{};
  a.logits = logits;
  a.topk_ids = topk_ids;
  a.gates = gates;
  a.dgates = dgates;
  a.dlosses = dlosses;
  a.lse = const_cast<float*>(lse);
  a.counts = const_cast<int32_t*>(counts);
  a.tokens = const_cast<int32_t*>(tokens);
  a.seg_offsets = seg_offsets;
  a.T = T;
  a.E = E;
  a.topk = topk;
  a.S = S;
  a.dlogits = dlogits;
  return mxf::launch_route_backward(a, logits_dtype == MXF_BF16, as_stream(stream)) ? MXF_ERR_LAUNCH : MXF_OK;
}

int moe_combine_backward(const void* dout, int dout_dtype, const void* y, int y_dtype, int64_t y_rows,
                         const float* gates, const int32_t* pair_row, int64_t T, int32_t topk, int64_t H, void* dy,
                         float* dgates, mxf_stream stream) {
  if (!valid_dtype(dout_dtype) || !valid_dtype(y_dtype)) return MXF_ERR_FORMAT;
  if (T < 0 || y_rows < 0 || topk < 1 || topk > 8 || H <= 0 || H % 8 != 0) return MXF_ERR_SHAPE;
  if (T > kMaxRows || T * (int64_t)topk > kMaxRows || y_rows > kMaxRows || H > kMaxRows) return MXF_ERR_UNSUPPORTED;
  const int64_t groups = T * mxf::cdiv(topk, mxf::combine_backward_pairs(T, topk));
  if (groups * mxf::combine_backward_threads(H, dout_dtype == MXF_BF16 && y_dtype == MXF_BF16) > mxf::kMaxThreads) return MXF_ERR_UNSUPPORTED;
  if (T == 0 || (y_rows == 0 && !dgates)) return MXF_OK;  // (a dy of no rows has no address)
  if (!dout || !gates || !pair_row || (!dy && !dgates) || (dgates && !y && y_rows > 0)) return MXF_ERR_NULL;
  const void* ptrs[] = {dout, y, gates, pair_row, dy, dgates};
  if (!all_aligned16(ptrs)) return MXF_ERR_ALIGN;
  mxf::CombineBackwardArgs a{dout, y, gates, pair_row, T, H, y_rows, topk, dy, dgates};
  return mxf::launch_combine_backward(a, y_dtype == MXF_BF16, dout_dtype == MXF_BF16, as_stream(stream)) ? MXF_ERR_LAUNCH
                                                                                                         : MXF_OK;
}

size_t nvfp4_tensor_scale_workspace_bytes(int64_t n, int x_dtype) {
  if (n <= 0 || !valid_dtype(x_dtype)) return 0;
  return mxf::amax_blocks(n / (x_dtype == MXF_BF16 ? 8 : 4)) > 1 ? mxf::kAmaxBlocks * sizeof(uint32_t) : 0;
}

int nvfp4_tensor_scale(const void* x, int x_dtype, int64_t n, float* scale, void* workspace, size_t workspace_bytes,
                       mxf_stream stream) {
  if (!valid_dtype(x_dtype)) return MXF_ERR_FORMAT;
  if (n <= 0 || n % 32 != 0) return MXF_ERR_SHAPE;
  if (!x || !scale) return MXF_ERR_NULL;
  if (!aligned16(x) || !aligned4(scale) || !aligned16(workspace)) return MXF_ERR_ALIGN;
  const size_t need = nvfp4_tensor_scale_workspace_bytes(n, x_dtype);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MXF_ERR_WORKSPACE;
  return mxf::launch_nvfp4_tensor_scale(x, x_dtype == MXF_BF16, n / (x_dtype == MXF_BF16 ? 8 : 4), scale,
                                        static_cast<uint32_t*>(workspace), as_stream(stream))
             ? MXF_ERR_LAUNCH
             : MXF_OK;
}

int fp4_quantize(const void* x, int x_dtype, int64_t rows, int64_t cols, int fmt, const float* tensor_scale,
                 const uint8_t* rnd, uint8_t* q, uint8_t* q_scale, uint8_t* qt, uint8_t* qt_scale, mxf_stream stream) {
  if (!valid_dtype(x_dtype) || !valid_weight(fmt)) return MXF_ERR_FORMAT;
  if (rows < 0 || cols <= 0 || cols % 32 != 0 || (tensor_scale && fmt == MXF_W_MXFP4)) return MXF_ERR_SHAPE;
  if (rows > kMaxRows || cols >= (int64_t(1) << 22)) return MXF_ERR_UNSUPPORTED;  // 32-bit offsets in 128 rows
  // workgroups of 512 threads per 128 x 128 values, or of 256 per 4096 (fp32) or 8192 (bf16) of them
  const int64_t threads = qt ? mxf::cdiv(mxf::cdiv(rows, 128) * mxf::cdiv(cols, 128), 8) * 8 * 512
                             : mxf::cdiv(rows * cols, x_dtype == MXF_BF16 ? 8192 : 4096) * 256;
  if (threads > mxf::kMaxThreads) return MXF_ERR_UNSUPPORTED;
  if (rows == 0) return MXF_OK;
  if (!x || (!q && !qt) || (q == nullptr) != (q_scale == nullptr) || (qt == nullptr) != (qt_scale == nullptr))
    return MXF_ERR_NULL;
  const void* ptrs[] = {x, rnd, q, q_scale, qt, qt_scale};
  if (!all_aligned16(ptrs) || !aligned4(tensor_scale)) return MXF_ERR_ALIGN;
  mxf::Fp4QuantArgs a{x, rows, cols, tensor_scale, rnd, q, q_scale, qt, qt_scale};
  return mxf::launch_fp4_quantize(a, x_dtype == MXF_BF16, fmt == MXF_W_NVFP4, as_stream(stream)) ? MXF_ERR_LAUNCH : MXF_OK;
}

int fp4_dequantize(const uint8_t* q, const uint8_t* q_scale, int64_t rows, int64_t cols, int fmt,
                   const float* tensor_scale, void* out, int out_dtype, mxf_stream stream) {
  if (!valid_weight(fmt) || !valid_dtype(out_dtype)) return MXF_ERR_FORMAT;
  if (rows < 0 || cols <= 0 || cols % 32 != 0 || (tensor_scale && fmt == MXF_W_MXFP4)) return MXF_ERR_SHAPE;
  if (rows > kMaxRows || cols > kMaxRows || mxf::cdiv(rows * cols, 4096) * 256 > mxf::kMaxThreads)
    return MXF_ERR_UNSUPPORTED;
  if (rows == 0) return MXF_OK;
  if (!q || !q_scale || !out) return MXF_ERR_NULL;
  const void* ptrs[] = {q, q_scale, out};
  if (!all_aligned16(ptrs) || !aligned4(tensor_scale)) return MXF_ERR_ALIGN;
  return mxf::launch_fp4_dequantize(q, q_scale, rows * (cols / 32), fmt == MXF_W_NVFP4, tensor_scale, out,
                                    out_dtype == MXF_BF16, as_stream(stream))
             ? MXF_ERR_LAUNCH
             : MXF_OK;
}

size_t fp4_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int fmt) {
  if (M <= 0 || N <= 0 || K <= 0 || !valid_weight(fmt)) return 0;
  return round_up(mxf::fp4_pair_workspace(M, N, K, fmt == MXF_W_NVFP4), 256);
}

int fp4_gemm(const uint8_t* a, const uint8_t* a_scale, int64_t M, const uint8_t* b, const uint8_t* b_scale, int64_t N,
             int64_t K, int fmt, const float* a_tensor_scale, const float* b_tensor_scale, void* c, int c_dtype,
             void* workspace, size_t workspace_bytes, mxf_stream stream) {
  if (!valid_weight(fmt) || !valid_dtype(c_dtype)) return MXF_ERR_FORMAT;
  if (M < 0 || N <= 0 || N % 16 != 0 || K <= 0 || K % 128 != 0) return MXF_ERR_SHAPE;
  if (fmt == MXF_W_MXFP4 && (a_tensor_scale || b_tensor_scale)) return MXF_ERR_SHAPE;
  // 32-bit byte offsets inside a tile of 256 rows; items and threads of a launch counted in 32 bits
  if (M > kMaxRows || N > kMaxRows || K >= (int64_t(1) << 24)) return MXF_ERR_UNSUPPORTED;
  if (mxf::cdiv(M, 128) * mxf::cdiv(N, 128) > mxf::kMostTiles || M * N >= (int64_t(1) << 34)) return MXF_ERR_UNSUPPORTED;
  if (M == 0) return MXF_OK;
  if (!a || !a_scale || !b || !b_scale || !c) return MXF_ERR_NULL;
  const void* ptrs[] = {a, a_scale, b, b_scale, c, workspace};
  if (!all_aligned16(ptrs) || !aligned4(a_tensor_scale) || !aligned4(b_tensor_scale)) return MXF_ERR_ALIGN;
  const size_t need = fp4_gemm_workspace_bytes(M, N, K, fmt);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MXF_ERR_WORKSPACE;
  return mxf::launch_fp4_pair(a, a_scale, M, b, b_scale, N, K, fmt == MXF_W_NVFP4, a_tensor_scale, b_tensor_scale, c,
                              c_dtype == MXF_BF16, workspace, as_stream(stream))
             ? MXF_ERR_LAUNCH
             : MXF_OK;
}

// The tile and K slices of a call of these sizes, as the launcher has them (for tests and profiles)
int mxf_fp4_pair_plan(int64_t M, int64_t N, int64_t K, int fmt, int32_t* out) {
  const mxf::Fp4PairPlan p = mxf::fp4_pair_plan(M, N, K, fmt == MXF_W_NVFP4);
  out[0] = p.bm;
  out[1] = p.bn;
  out[2] = p.slices;
  return 3;
}

}  // extern "C"
