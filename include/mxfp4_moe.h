/*
 * mxfp4_moe.h - C ABI of the MI355X (gfx950) MXFP4 mixture-of-experts expert path.
 *
 * The library computes the hot path of a DeepSeek-V4-Flash-style MoE layer whose
 * routed-expert weights are MXFP4: E2M1 codes (1 sign / 2 exponent / 1 mantissa
 * bit) with one UE8M0 scale per 32 K-elements, fed to block-scaled matrix
 * instructions without dequantisation to a 16-bit type
 * (page "DGX Spark 原生 FP4 矩阵指令：DwarfStar 如何利用 Blackwell 加速推理",
 * sections 一 and 二). Each token goes to the top-6 of 256 experts and runs two
 * FC contractions per expert (page "【DeepSeek V4】Triton FP4 优化实战：近距离感受
 * 老黄的刀法", "FP4 MoE GEMM 是什么？"); SwiGLU and the FP8 requantisation are
 * fused between them (page "Domestic GPUs are awesome! Moore thread full-link
 * adaptation DeepSeek-V4": "SwiGLU + FP8 quant", routing, dispatch/combine).
 *
 * Conventions shared by every entry point:
 *  - Pointers are DEVICE pointers to caller-owned, contiguous, row-major buffers.
 *    The library never allocates, frees, copies to the host or synchronises.
 *  - Every call is asynchronous on `stream` (a hipStream_t; NULL = the legacy
 *    default stream). Nothing is read back to the host: counts and offsets stay
 *    on the device.
 *  - Every argument is validated before anything is enqueued. On any error the
 *    function returns a non-zero mxf_status and enqueues nothing (no silent
 *    fallback to another path - the pages' FP4 path errors out on a K it cannot
 *    take, page "DGX Spark 原生 FP4 矩阵指令" section 三). MXF_ERR_LAUNCH means a
 *    launch failed after validation; device faults surface at the caller's next
 *    synchronisation.
 *  - Byte layouts:
 *      E4M3 activations   [rows][K]     u8, one OCP E4M3FN code per element
 *      E2M1 activations   [rows][K/2]   u8, element 2n in the low nibble of byte n
 *                                           (page "【DeepSeek V4】Triton FP4 优化实战",
 *                                           "第二步": even column = low nibble)
 *      UE8M0 scales       [rows][K/32]  u8, value 2^(byte - 127)
 *      MXFP4 weights      [N][K/2] codes + [N][K/32] scales, K contiguous ("nt")
 *  - Quantisation rule (OCP MX): per 32-element block, scale byte =
 *    clamp(floor(log2 amax) - emax + 127, 0, 254) (0 when amax = 0; emax = 8 for
 *    E4M3, 2 for E2M1), elements rounded to nearest even on the element grid,
 *    saturating at the largest normal (448 / 6), sign kept.
 *  - Alignment: every code and scale pointer must be 16-byte aligned, every
 *    fp32/bf16 pointer 16-byte aligned (128-bit loads and stores).
 */
#ifndef MXFP4_MOE_H
#define MXFP4_MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MXF_OK = 0,
  MXF_ERR_NULL = 1,        /* a required pointer is NULL */
  MXF_ERR_SHAPE = 2,       /* a size is negative, or not a multiple the kernels need */
  MXF_ERR_ALIGN = 3,       /* a pointer is not 16-byte aligned */
  MXF_ERR_FORMAT = 4,      /* unknown element format or dtype enum */
  MXF_ERR_UNSUPPORTED = 5, /* valid arguments outside the sizes this library handles */
  MXF_ERR_LAUNCH = 6,      /* a kernel launch failed (hipGetLastError) */
  MXF_ERR_WORKSPACE = 7    /* workspace missing or smaller than required */
} mxf_status;

typedef enum { MXF_E4M3 = 0, MXF_E2M1 = 1 } mxf_elem;   /* activation element format */
typedef enum { MXF_F32 = 0, MXF_BF16 = 1 } mxf_dtype;   /* floating-point buffer type */

typedef void* mxf_stream; /* a hipStream_t */

/* Human-readable name of a status code (static storage, never NULL). */
const char* mxf_status_str(int status);

/* ABI version of this header (bumped on any signature change). */
int mxf_abi_version(void);
#define MXF_ABI_VERSION 2

/*
 * mxfp4_quantize_act - quantise activation rows per 32-element block.
 * Defined by: the activation side of the FP4 path, page "DGX Spark 原生 FP4 矩阵
 * 指令" sections 一 (E2M1 elements with one UE8M0 scale per block, fed to the
 * matrix instruction as they are) and 二 (activations kept in FP4 end to end on the
 * FP4 path); the FP8 activations of the grouped FP8 x FP4 GEMM, page "【DeepSeek
 * V4】Triton FP4 优化实战" section 第零步 (the profiled m_grouped_fp8_fp4 call); and
 * the "FP8 quant" step of page "Domestic GPUs are awesome! ... DeepSeek-V4". The
 * block rule itself (floor(log2 amax) - emax, round to nearest even) is the OCP MX
 * one stated at the top of this header.
 *   x        [rows][K] bf16 (x_dtype = MXF_BF16) or fp32 (MXF_F32) values
 *   fmt      MXF_E4M3 -> q [rows][K] ; MXF_E2M1 -> q [rows][K/2] (packed)
 *   q_scale  [rows][K/32] UE8M0 bytes
 * Bit-exact with the OCP MX rule above. Requires K % 32 == 0; rows == 0 is a
 * no-op. Errors: NULL, SHAPE (K % 32, negative sizes), FORMAT, ALIGN.
 */
int mxfp4_quantize_act(const void* x, int x_dtype, int64_t rows, int64_t K, int fmt,
                       uint8_t* q, uint8_t* q_scale, mxf_stream stream);

/*
 * mxfp4_gemm - dense MXFP4 GEMM, C = A_hat * W_hat^T
 * Defined by: the dense MXFP4 entry of page "DGX Spark 原生 FP4 矩阵指令" section 二,
 * the K-shape guard of its section 三 (a K the kernels cannot take is an error, never
 * a silent other path), and the dense shapes of the accuracy table in page "【DeepSeek
 * V4】Triton FP4 优化实战" section 第二步 (16 x 32 x 4096 and 64 x 4096 x 7168).
 *   a        [M][K] bf16 activations, quantised inside the call per 32-block to
 *            act_fmt (E4M3 or E2M1) with the rule above. For M <= 16 the GEMM
 *            kernel quantises them in registers and the codes are never written;
 *            for larger M the quantised copy lives only in `workspace`
 *   w        [N][K/2] E2M1 codes, w_scale [N][K/32] UE8M0
 *   c        [M][N] fp32 output (fp32 accumulation of exact products)
 *   workspace, workspace_bytes: device scratch of at least
 *            mxfp4_gemm_workspace_bytes(M, N, K, act_fmt) bytes (16-byte
 *            aligned; may be NULL when that is 0): the quantised activations
 *            (M > 16) and the fp32 partial sums of the K slices (M <= 64 with a
 *            long K; for M <= 16 only when the weight codes exceed 1 MiB - below
 *            that the call is one launch and needs no workspace); its contents on
 *            entry are ignored and on exit undefined. The slice sums are added in
 *            a fixed order, so results are bit-identical from run to run.
 * Requires K % 512 == 0 (one 512-k super-step of scaled-MFMA K steps) and
 * N % 16 == 0; M >= 0 (M == 0 is a no-op). For M > 64 with N % 256 == 0 (the
 * tiled kernels) the quantised activations and the weight codes must each stay
 * below 4 GiB, else UNSUPPORTED; otherwise (the weight-streaming kernel) 64
 * weight rows must stay below 4 GiB (K < 2^27), else UNSUPPORTED.
 * Errors: NULL, SHAPE, ALIGN, FORMAT, WORKSPACE, UNSUPPORTED.
 */
size_t mxfp4_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int act_fmt);
int mxfp4_gemm(const uint16_t* a, int64_t M, int64_t N, int64_t K, int act_fmt,
               const uint8_t* w, const uint8_t* w_scale, float* c,
               void* workspace, size_t workspace_bytes, mxf_stream stream);

/*
 * mxfp4_gemm_noalloc - mxfp4_gemm with its workspace inside the library.
 * For callers that cannot allocate device memory or pass a workspace: code under
 * HIP graph capture, tight serving loops, harnesses that forbid allocation. The
 * result is that of mxfp4_gemm (the same kernels, bit for bit).
 *   The workspace is a fixed device array of MXF_NOALLOC_SCRATCH_BYTES (16 MiB) per
 *   GPU, held from the library's first use on that GPU until the process ends; its
 *   device address is looked up once per device on the first call made with that
 *   device current. Nothing is allocated or freed by any call.
 *   Every call on one GPU shares that GPU's array: calls that overlap in time on one
 *   GPU (different streams, or different host threads) race and give undefined
 *   results; calls ordered on one stream are safe. Nothing in the array needs to
 *   start at zero (each call overwrites what it reads).
 * Arguments as for mxfp4_gemm without the workspace pair. A call whose workspace
 * (mxfp4_gemm_workspace_bytes) exceeds the array returns MXF_ERR_WORKSPACE before
 * touching the device (the 64 x 4096 x 7168 GEMM needs 4.5 MiB). Other errors as
 * for mxfp4_gemm; MXF_ERR_LAUNCH also if the array's address cannot be found.
 */
#define MXF_NOALLOC_SCRATCH_BYTES ((size_t)16 << 20)
size_t mxfp4_noalloc_scratch_bytes(void);
int mxfp4_gemm_noalloc(const uint16_t* a, int64_t M, int64_t N, int64_t K, int act_fmt,
                       const uint8_t* w, const uint8_t* w_scale, float* c, mxf_stream stream);

/*
 * mxfp4_gemm_w4a16 / nvfp4_gemm_w4a16 - FP4 weights x bf16 activations:
 *   C[M][N] (fp32) = A . W_hat^T, A [M][K] bf16 used as given (no activation
 *   quantisation), fp32 accumulation.
 * Defined by: the fused dequantise + matmul of page "【DeepSeek V4】Triton FP4 优化实战"
 * section 第二步 (packed FP4 weights, even column in the low nibble, turned into bf16
 * inside the kernel and multiplied in bf16, no 16-bit weight copy in memory), with its
 * accuracy table's shapes (1 x 32 x 4096, 1 x 4096 x 7168, 64 x 4096 x 7168); the
 * NVFP4 block format is the one of the kind::mxf4nvf4 / scale_vec::4X instruction of page
 * "DGX Spark 原生 FP4 矩阵指令" section 一 (E2M1 codes, a UE4M3 scale per 16 elements).
 *   w        [N][K/2] E2M1 codes, element 2n in the low nibble of byte n
 *   w_scale  mxfp4: [N][K/32] UE8M0 bytes, value 2^(byte - 127), bytes 2 .. 252 (every
 *            decoded weight then lies in bf16's normal range; smaller bytes give weights
 *            the bf16 instruction may flush, larger ones overflow bf16);
 *            nvfp4: [N][K/16] UE4M3 bytes (OCP E4M3 with the sign bit clear), value
 *            2^(e-7) (1 + m/8), or m 2^-9 for e = 0; 0x7F (NaN) is not a valid scale
 *   c        [M][N] fp32
 *   workspace, workspace_bytes: device scratch of at least fp4_w4a16_workspace_bytes(M,
 *            N, K) bytes (0 means none needed; 16-byte aligned): fp32 partial sums of
 *            the K slices, added in a fixed order (bit-identical results run to run).
 * Every weight value code x scale is exact in bf16, so the only rounding is the fp32
 * accumulation. Requires K % 512 == 0, N % 16 == 0, M >= 0 (0 is a no-op), K < 2^27.
 * Errors: NULL, SHAPE, ALIGN, WORKSPACE, UNSUPPORTED.
 */
size_t fp4_w4a16_workspace_bytes(int64_t M, int64_t N, int64_t K);
int mxfp4_gemm_w4a16(const uint16_t* a, int64_t M, int64_t N, int64_t K, const uint8_t* w,
                     const uint8_t* w_scale, float* c, void* workspace, size_t workspace_bytes,
                     mxf_stream stream);
int nvfp4_gemm_w4a16(const uint16_t* a, int64_t M, int64_t N, int64_t K, const uint8_t* w,
                     const uint8_t* w_scale, float* c, void* workspace, size_t workspace_bytes,
                     mxf_stream stream);

/*
 * q8_quantize_act / mxfp4_gemm_q8 - the lookup-table route: Q8 activations x MXFP4
 * weights through int8 products.
 * Defined by: the generic FP4 path of hardware without FP4 matrix instructions, page
 * "DGX Spark 原生 FP4 矩阵指令" sections 二 and 三 (FP4 weights expanded to Q8-style
 * integers, Q8_1-style activations, lossless and with no FP4 speed bonus); the Q8_0
 * block (32 int8 + an fp16 scale) and the exact FP4 <-> 4-bit lookup-table equivalence,
 * page "企业官网建设流程全解析" sections 四 and 五.
 * q8_quantize_act:
 *   x  [rows][K] bf16; q [rows][K] int8; d [rows][K/32] fp16 (2-byte aligned)
 *   per 32-block: d = fp16(amax / 127) (fp32 quotient, round to nearest even),
 *   q = clamp(round_to_nearest_even(x / d), -127, 127) with the quotient in fp32, and
 *   q = 0 where d = 0. Bit-exact. Requires K % 32 == 0. Errors: NULL, SHAPE, ALIGN.
 *   (Q8_1's second per-block number, d times the sum of q, serves asymmetric weight
 *   formats; E2M1 is symmetric, so it is not formed.)
 * mxfp4_gemm_q8:
 *   C[M][N] (fp32) = sum over 32-blocks b of (sum_k q[m][k] w8[n][k]) d[m][b] 2^(e - 128)
 *   where w8 = 2 x e2m1(code) in {0, +-1, +-2, +-3, +-4, +-6, +-8, +-12} (a 16-entry table)
 *   and e the weight's UE8M0 byte (bytes 2 .. 252): w8 2^(e - 128) is the MXFP4 weight
 *   exactly. Each block's integer sum is exact; the scaling and the sum over blocks
 *   round in fp32. q, d as written by q8_quantize_act (d 16-byte aligned here); w, w_scale
 *   as for mxfp4_gemm; workspace >= mxfp4_gemm_q8_workspace_bytes(M, N, K) (K-slice
 *   partial sums, added in a fixed order). Requires K % 512 == 0, N % 16 == 0,
 *   K < 2^27. Errors: NULL, SHAPE, ALIGN, WORKSPACE, UNSUPPORTED.
 */
int q8_quantize_act(const uint16_t* x, int64_t rows, int64_t K, int8_t* q, uint16_t* d, mxf_stream stream);
size_t mxfp4_gemm_q8_workspace_bytes(int64_t M, int64_t N, int64_t K);
int mxfp4_gemm_q8(const int8_t* q, const uint16_t* d, int64_t M, int64_t N, int64_t K, const uint8_t* w,
                  const uint8_t* w_scale, float* c, void* workspace, size_t workspace_bytes, mxf_stream stream);

/*
 * moe_route_permute - top-k routing and the expert-grouped permutation.
 * Defined by: page "【DeepSeek V4】Triton FP4 优化实战" section "FP4 MoE GEMM 是什么？"
 * (each token picks 6 of 256 experts) and page "Domestic GPUs are awesome! ...
 * DeepSeek-V4" (MoE routing / Top-k as an operator, and the dispatch that groups a
 * token's rows by expert before the expert GEMMs); the grouped, row-contiguous
 * layout is the one of the profiled m_grouped_..._contiguous call in the Triton
 * page's section 第零步.
 *   logits         [T][E] fp32
 *   topk_ids       [T][topk] i32: per token the topk largest logits, distinct
 *                  experts, ordered by (logit descending, expert index ascending)
 *   gates          [T][topk] fp32: softmax over the selected logits
 *                  (exp(l_j - l_0) / sum_j' exp(l_j' - l_0))
 *   expert_offsets [E+1] i32: exclusive prefix sum of per-expert pair counts
 *   sorted_pair    [T*topk] i32: pairs p = t*topk + j grouped by expert,
 *                  ascending p inside an expert (stable)
 *   pair_row       [T*topk] i32: inverse of sorted_pair
 * The integer outputs are bit-exact (deterministic). sorted_pair is also used
 * as scratch while the call runs. Requires 1 <= topk <= min(E, 8), E <= 1024,
 * T*topk < 2^31; T == 0 writes only expert_offsets (all zero). Errors: NULL,
 * SHAPE, ALIGN, UNSUPPORTED.
 */
int moe_route_permute(const float* logits, int64_t T, int32_t E, int32_t topk,
                      int32_t* topk_ids, float* gates, int32_t* expert_offsets,
                      int32_t* sorted_pair, int32_t* pair_row, mxf_stream stream);

/*
 * moe_quantize_route - mxfp4_quantize_act of the layer input and moe_route_permute
 * of its router logits in one launch, for decode-sized batches.
 * Defined by: the two calls above (the same steps, outputs bit-identical to them);
 * the two steps share no data, so one launch replaces two (at decode sizes a
 * launch's fixed cost is most of either step's time).
 *   x [T][H] bf16 or fp32 (x_dtype); logits [T][E] fp32
 *   q, q_scale     [T][H] (E4M3) or [T][H/2] (E2M1), [T][H/32], as mxfp4_quantize_act
 *   topk_ids, gates, expert_offsets, sorted_pair, pair_row   as moe_route_permute
 * Requires T <= 64 and E <= 256 (else UNSUPPORTED: use the two calls), H % 32 == 0,
 * 1 <= topk <= min(E, 8). expert_offsets is written (all zero) even when T == 0.
 * Errors: NULL, SHAPE, ALIGN, FORMAT, UNSUPPORTED.
 */
int moe_quantize_route(const void* x, int x_dtype, const float* logits, int64_t T, int64_t H,
                       int32_t E, int32_t topk, int act_fmt, uint8_t* q, uint8_t* q_scale,
                       int32_t* topk_ids, float* gates, int32_t* expert_offsets,
                       int32_t* sorted_pair, int32_t* pair_row, mxf_stream stream);

/*
 * moe_grouped_mxfp4_gemm - both expert FCs for every (token, expert) pair.
 * Defined by: page "DGX Spark 原生 FP4 矩阵指令" section 二 (the MoE MXFP4 entry;
 * weights stay FP4 into the matrix instruction), page "【DeepSeek V4】Triton FP4
 * 优化实战" sections "FP4 MoE GEMM 是什么？" (two FC per expert) and 第二步 (expert
 * FC1 is 4096 x 7168; even column in the low nibble), and page "Domestic GPUs are
 * awesome! ... DeepSeek-V4" ("SwiGLU + FP8 quant" fused between the two FCs).
 *   q, q_scale     quantised layer input [T][H] (E4M3) or [T][H/2] (E2M1) + [T][H/32]
 *   act_fmt        element format of q and of h
 *   expert_offsets, sorted_pair  as written by moe_route_permute
 *   w1, w1_scale   [E][2I][H/2], [E][2I][H/32]: rows 0..I-1 gate, I..2I-1 up
 *   w2, w2_scale   [E][H][I/2],  [E][H][I/32]
 *   h, h_scale     output workspace [T*topk][I] (E4M3) or [T*topk][I/2] (E2M1)
 *                  + [T*topk][I/32]: silu(gate) * up requantised per 32 along I
 *   y              [T*topk][H] fp32 or bf16 (y_dtype): FC2 output in the
 *                  permuted (expert-grouped) row order
 * Row r of the permuted order is token sorted_pair[r] / topk. The grid is sized
 * from T and topk; per-expert counts are read on the device.
 * Requires H % 512 == 0, I % 512 == 0, 1 <= topk <= min(E, 8), E <= 1024;
 * one expert's w1 and w2 codes must each stay below 4 GiB, and for T > 64 (the
 * tiled kernels) so must q and h, else UNSUPPORTED. T == 0 is a no-op.
 * Errors: NULL, SHAPE, ALIGN, FORMAT, UNSUPPORTED.
 */
int moe_grouped_mxfp4_gemm(const uint8_t* q, const uint8_t* q_scale, int act_fmt,
                           int64_t T, int32_t topk, int64_t H, int64_t I, int32_t E,
                           const int32_t* expert_offsets, const int32_t* sorted_pair,
                           const uint8_t* w1, const uint8_t* w1_scale,
                           const uint8_t* w2, const uint8_t* w2_scale,
                           uint8_t* h, uint8_t* h_scale,
                           void* y, int y_dtype, mxf_stream stream);

/*
 * moe_grouped_mxfp4_gemm_combine - both expert FCs with FC2 fused into the
 * gate-weighted combine, for decode-sized batches:
 *   out[t] = sum_{j=0..topk-1} gates[t][j] * (h_hat[r(t,j)] . W2_hat[e(t,j)]^T)
 * Defined by: the FC1 / SwiGLU / requantisation steps of moe_grouped_mxfp4_gemm
 * above, then the combine half of MoE dispatch/combine (page "Domestic GPUs are
 * awesome! ... DeepSeek-V4") applied inside the FC2 kernel, which the closing
 * lessons of page "【DeepSeek V4】Triton FP4 优化实战" motivate (cut the data moved
 * between steps, not the arithmetic). The FC2 products of one output column for
 * every (token, slot) pair stay in fp32 on the chip (y is never stored and never
 * rounded to bf16) and are summed in slot order j = 0, 1, ... with fused
 * multiply-adds, then stored as out_dtype (bf16: round to nearest even).
 *   q, q_scale, act_fmt, expert_offsets, sorted_pair, w1.., w2.., h, h_scale
 *                  as for moe_grouped_mxfp4_gemm (h is still written: FC2 reads it)
 *   topk_ids, pair_row, gates   [T][topk] int32, [T*topk] int32, [T][topk] fp32,
 *                  as written by moe_route_permute (FC1 reads the expert-grouped
 *                  order, the fused FC2 the token-major one)
 *   out            [T][H] fp32 or bf16 (out_dtype), caller-allocated
 * Requires T <= 64 (larger batches: moe_grouped_mxfp4_gemm + moe_unpermute_combine,
 * else UNSUPPORTED) and the shape rules of moe_grouped_mxfp4_gemm. Deterministic:
 * no atomics, fixed summation order. T == 0 is a no-op.
 * Errors: NULL, SHAPE, ALIGN, FORMAT, UNSUPPORTED.
 */
int moe_grouped_mxfp4_gemm_combine(const uint8_t* q, const uint8_t* q_scale, int act_fmt,
                                   int64_t T, int32_t topk, int64_t H, int64_t I, int32_t E,
                                   const int32_t* expert_offsets, const int32_t* sorted_pair,
                                   const int32_t* topk_ids, const int32_t* pair_row,
                                   const float* gates,
                                   const uint8_t* w1, const uint8_t* w1_scale,
                                   const uint8_t* w2, const uint8_t* w2_scale,
                                   uint8_t* h, uint8_t* h_scale,
                                   void* out, int out_dtype, mxf_stream stream);

/*
 * moe_unpermute_combine - out[t] = sum_{j=0..topk-1} gates[t][j] * y[pair_row[t*topk+j]]
 * Defined by: the combine half of MoE dispatch/combine, page "Domestic GPUs are
 * awesome! ... DeepSeek-V4"; the gates are the routing weights of page "【DeepSeek
 * V4】Triton FP4 优化实战" section "FP4 MoE GEMM 是什么？".
 * accumulated in fp32 in slot order j = 0, 1, ..., then stored as out_dtype
 * (bf16: round to nearest even). y [T*topk][H] (y_dtype), out [T][H].
 * Requires H % 8 == 0, T H below 2^35 and T topk below 2^31. Errors: NULL, SHAPE, ALIGN,
 * FORMAT, UNSUPPORTED.
 */
int moe_unpermute_combine(const void* y, int y_dtype, const float* gates,
                          const int32_t* pair_row, int64_t T, int32_t topk, int64_t H,
                          void* out, int out_dtype, mxf_stream stream);

/* FP4 weight formats of the calls that take both: E2M1 codes with one UE8M0 scale per 32
 * K-elements, or with one UE4M3 scale per 16 (as in nvfp4_gemm_w4a16). */
typedef enum { MXF_W_MXFP4 = 0, MXF_W_NVFP4 = 1 } mxf_weight;

/*
 * moe_grouped_gemm_w4a16 - ragged grouped GEMM of bf16 activations with FP4 expert weights:
 *   y[r] = a[src(r)] * W_hat_e^T   for every expert e and row r in
 *                                  [expert_offsets[e], expert_offsets[e+1])
 * the grouped form of mxfp4_gemm_w4a16 / nvfp4_gemm_w4a16: no activation quantisation,
 * products exact, fp32 accumulation. An expert may have any number of rows, none included.
 *   a            [a_rows][K] bf16
 *   sorted_pair  NULL: src(r) = r (a_rows must be R); else [R] int32 and src(r) =
 *                sorted_pair[r] / topk (as moe_route_permute writes it; topk is ignored
 *                when it is NULL). An entry outside [0, a_rows * topk) reads some row of a
 *                or zeros, never anything else.
 *   expert_offsets [E+1] int32, ascending, within [0, R]; values outside are held to it
 *   w, w_scale   [E][N][K/2] codes, [E][N][K/32] UE8M0 (bytes 2..252) or [E][N][K/16] UE4M3
 *   swiglu       0: y [R][N]; 1: rows 0..N/2-1 of W are gate rows, the others the up rows,
 *                and y [R][N/2] = silu(gate) * up, in fp32 before the one rounding to y_dtype
 *   y            fp32 or bf16 (y_dtype; round to nearest even). Rows of y outside
 *                [expert_offsets[0], expert_offsets[E]) are left as they were.
 * Deterministic: no atomics, and the same call sums in the same order (which kernel an expert
 * runs in, and with it the order, follows from R, E, N, K and its own rows); a row's result does
 * not depend on what other rows hold. Requires K % 128 == 0, N % 16 == 0 (swiglu: N % 32 == 0),
 * E <= 1024, and the bytes of one expert's codes below 4 GiB with a margin of 257 rows;
 * with sorted_pair also a below 4 GiB; and fewer than 2^24 workgroups a launch, which E N below
 * 2^30 with R N below 2^38 keeps to. R == 0 is a no-op.
 * Errors: NULL, SHAPE, ALIGN, FORMAT, UNSUPPORTED.
 */
int moe_grouped_gemm_w4a16(const uint16_t* a, int64_t a_rows, int64_t R, const int32_t* sorted_pair, int32_t topk,
                           const int32_t* expert_offsets, int32_t E, int64_t N, int64_t K, int w_fmt,
                           const uint8_t* w, const uint8_t* w_scale, int swiglu, void* y, int y_dtype,
                           mxf_stream stream);

/*
 * fp4_gemm_w4a16_lora - a shared FP4 projection with the low-rank adapters of many requests:
 *   c[t] = a[t] * W_hat^T + scaling[l] * (a[t] * lora_a[l]^T) * lora_b[l]^T
 * where l = seg_adapter[s] for the segment s with seg_offsets[s] <= t < seg_offsets[s+1].
 * A segment whose adapter is outside [0, L) (say -1), and rows in no segment, get the
 * projection alone. Infinities and NaN of an adapter reach the rows of its segments only.
 *   a            [M][K] bf16;  w, w_scale as for mxfp4_gemm_w4a16 / nvfp4_gemm_w4a16
 *   seg_offsets  [S+1] int32, ascending (a request's rows are consecutive); seg_adapter [S]
 *   lora_a       [L][rank][K] bf16;  lora_b [L][N][rank] bf16;  scaling [L] fp32. An adapter
 *                of a smaller rank is padded with zero rows of lora_a.
 *   c            [M][N] fp32 or bf16 (c_dtype), one rounding at the end; between its
 *                two factors the low-rank product is held in fp32
 *   workspace    fp4_w4a16_lora_workspace_bytes() bytes, 16-byte aligned, contents
 *                irrelevant; calls that may overlap need one each
 * Requires K % 512 == 0, N % 16 == 0, rank % 8 == 0, 8 <= rank <= 128, and the codes and one
 * adapter's lora_b below 4 GiB (with a margin of 257 rows), M < 2^28 and M N below 2^38. S == 0 (with L == 0
 * or not): the projection alone. M == 0 is a no-op.
 * Errors: NULL, SHAPE, ALIGN, FORMAT, UNSUPPORTED, WORKSPACE.
 */
size_t fp4_w4a16_lora_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t rank);
int fp4_gemm_w4a16_lora(const uint16_t* a, int64_t M, int64_t N, int64_t K, int w_fmt, const uint8_t* w,
                        const uint8_t* w_scale, const int32_t* seg_offsets, const int32_t* seg_adapter, int32_t S,
                        const uint16_t* lora_a, const uint16_t* lora_b, const float* scaling, int32_t L,
                        int32_t rank, void* c, int c_dtype, void* workspace, size_t workspace_bytes,
                        mxf_stream stream);

/*
 * moe_block_norm - the step between two blocks of a decoder layer, one pass over each row:
 *   b = y[t], or with topk > 0 the combine sum_j expert_gates[t][j] * y[pair_row[t*topk+j]]
 *       (fp32, slot order, as moe_unpermute_combine; an entry of pair_row outside
 *       [0, y_rows) is a dropped pair and adds nothing)
 *   p = post_weight * b / sqrt(mean(b^2) + eps)   (post_weight NULL: p = b)
 *   r = residual_scale * x[t] + gate * p          (x NULL: r = gate * p)
 *   n = pre_weight * r / sqrt(mean(r^2) + eps)    (pre_weight NULL: weights of one)
 *   q, q_scale = n quantised as by mxfp4_quantize_act (from the fp32 n)
 * All in fp32; each result is rounded once, when it is stored.
 *   y            [T][H], or with topk > 0 [y_rows][H] (y_dtype)
 *   x, r         [T][H] (x_dtype, both); r may be x itself
 *   post_weight, pre_weight  [H] (weight_dtype)
 *   gate         gate_mode 0: none (gate ignored), 1: [H], 2: [T], 3: [T][H] (gate_dtype)
 *   r, n, q      any may be NULL (not wanted), not all; n [T][H] (n_dtype); q [T][H] (E4M3)
 *                or [T][H/2] (E2M1) by fmt, with q_scale [T][H/32]
 * Requires H % 8 == 0 (H % 32 == 0 with q), H <= 65536, eps > 0, topk <= 8; with topk == 0
 * y_rows must be T, with topk > 0 at least 1. T == 0 is a no-op.
 * Errors: NULL, SHAPE, ALIGN, FORMAT, UNSUPPORTED.
 */
int moe_block_norm(const void* y, int y_dtype, int64_t y_rows, const float* expert_gates, const int32_t* pair_row,
                   int32_t topk, int64_t T, int64_t H, const void* x, int x_dtype, float residual_scale,
                   const void* post_weight, const void* pre_weight, int weight_dtype, float eps, const void* gate,
                   int gate_dtype, int gate_mode, void* r, void* n, int n_dtype, int fmt, uint8_t* q,
                   uint8_t* q_scale, mxf_stream stream);

/*
 * moe_balance_loss - the load-balance and z losses of a router, with its per-expert counts.
 * With p = softmax(logits[t]) over all E experts, lse = log(sum exp(logits[t])), sequences s =
 * [seg_offsets[s], seg_offsets[s+1]), n_s its tokens that count, n = sum n_s, S' the sequences with
 * n_s > 0, c_si the pairs of those tokens that go to expert i, P_si = 1/n_s sum_t p_ti:
 *   losses[0] = 1/S' sum_s E / (topk n_s) sum_i c_si P_si    (1 where both are spread evenly)
 *   losses[1] = 1/n sum_t lse_t^2
 * Both are 0 where no token counts. A token counts if it is in a sequence, token_mask does not
 * exclude it and one of its logits at least is not -inf (experts ruled out hold -inf: p = 0).
 *   logits       [T][E] fp32 or bf16 (logits_dtype)
 *   topk_ids     [T][topk] int32 as moe_route_permute writes them; an id outside [0, E) is a
 *                dropped pair and counts for nothing, the same id twice counts twice
 *   token_mask   [T] bytes, 0 excludes the token (any alignment); NULL: none excluded
 *   seg_offsets  [S+1] int32, ascending within [0, T] (values outside are held to it; empty
 *                sequences are fine); NULL: one sequence of all tokens, S must be 1
 *   counts       [S][E] int32: c;  prob_mean [S][E] fp32: P (0 in an empty sequence)
 *   tokens       [S+2] int32: n_s, then n, then S'
 *   lse          [T] fp32, -inf for a token that does not count (the gradient reads it)
 *   losses       [2] fp32
 *   workspace    moe_balance_loss_workspace_bytes(T, E, S) bytes (0: none needed, may be NULL),
 *                16-byte aligned, contents irrelevant; calls that may overlap need one each
 * Sums in fp32 and above in a fixed order: deterministic. NaN and +inf logits make the losses NaN.
 * Requires 1 <= topk <= min(E, 8), E <= 1024, S >= 1, T topk below 2^31, T below 2^26 and
 * S ceil(E / 64) below 2^23. T == 0 writes zeros. Errors: NULL, SHAPE, ALIGN, FORMAT, UNSUPPORTED,
 * WORKSPACE.
 */
size_t moe_balance_loss_workspace_bytes(int64_t T, int32_t E, int32_t S);
int moe_balance_loss(const void* logits, int logits_dtype, const int32_t* topk_ids, const uint8_t* token_mask,
                     const int32_t* seg_offsets, int32_t S, int64_t T, int32_t E, int32_t topk, int32_t* counts,
                     int32_t* tokens, float* prob_mean, float* lse, float* losses, void* workspace,
                     size_t workspace_bytes, mxf_stream stream);

/*
 * moe_route_backward - the gradient of the logits, from the gates' and the losses':
 *   dlogits[t][i] = sum_{j: topk_ids[t][j] = i} gates[t][j] (dgates[t][j] - sum_k gates[t][k] dgates[t][k])
 *     + dlosses[0] E / (S' topk n_s^2) p_i (c_si - sum_j p_j c_sj) + dlosses[1] 2/n lse p_i
 * (the first line: the softmax over the selected logits of moe_route_permute; the second for tokens
 * that count, with the counts held constant).
 *   gates, dgates [T][topk] fp32; dgates NULL: no such term (gates and topk_ids are ignored)
 *   dlosses      [2] fp32 on the device (4-byte aligned); NULL: no such terms (logits, lse, counts,
 *                tokens and seg_offsets are ignored)
 *   lse, counts, tokens  as moe_balance_loss wrote them for these sequences. Where each sequence's tokens lie
 *                on several GPUs, the losses of them all take counts, n_s and n added up over the GPUs;
 *                S' (the last of tokens) is then the number of n_s > 0 after that, not a sum
 *   dlogits      [T][E], of logits_dtype; every value is written
 * Sizes as for moe_balance_loss. T == 0 is a no-op. Errors: NULL (neither term wanted, too), SHAPE,
 * ALIGN, FORMAT, UNSUPPORTED.
 */
int moe_route_backward(const void* logits, int logits_dtype, const int32_t* topk_ids, const float* gates,
                       const float* dgates, const float* dlosses, const float* lse, const int32_t* counts,
                       const int32_t* tokens, const int32_t* seg_offsets, int32_t S, int64_t T, int32_t E, int32_t topk,
                       void* dlogits, mxf_stream stream);

/*
 * moe_combine_backward - the gradient of moe_unpermute_combine, p = t topk + j:
 *   dy[pair_row[p]] = gates[p] * dout[t],   dgates[p] = sum_h dout[t][h] * y[pair_row[p]][h]
 * in fp32, each result rounded once when it is stored.
 *   dout         [T][H] fp32 or bf16 (dout_dtype);  y, dy [y_rows][H] (y_dtype)
 *   pair_row     [T*topk] int32; an entry outside [0, y_rows) is a dropped pair (its dgates is 0).
 *                The others name a row each, no row twice. Rows of dy that none names are left as
 *                they were.
 *   dy, dgates   either may be NULL (not wanted), not both; y may be NULL without dgates
 * dy may be y itself. Requires H % 8 == 0, topk <= 8, T topk below 2^31, and T (or T topk below 256
 * tokens) workgroups of at most 512 threads below 2^32 threads. T == 0 is a no-op.
 * Errors: NULL, SHAPE, ALIGN, FORMAT, UNSUPPORTED.
 */
int moe_combine_backward(const void* dout, int dout_dtype, const void* y, int y_dtype, int64_t y_rows,
                         const float* gates, const int32_t* pair_row, int64_t T, int32_t topk, int64_t H, void* dy,
                         float* dgates, mxf_stream stream);

/*
 * nvfp4_tensor_scale - the scale of a whole tensor for NVFP4: the smallest power of two g (at least
 * 2^-126) with max |x| <= 6 * 448 * g, and 1 for a tensor of zeros. A power of two, so that block scale
 * times g, and with it every quantised value, is exact.
 *   x  n values, fp32 or bf16 (n % 32 == 0, not 0);  scale [1] fp32 on the device (4-byte aligned)
 *   workspace    nvfp4_tensor_scale_workspace_bytes(n, x_dtype) bytes (0: none needed, may be NULL),
 *                16-byte aligned, contents irrelevant; calls that may overlap need one each
 * Errors: NULL, SHAPE, ALIGN, FORMAT, WORKSPACE.
 */
size_t nvfp4_tensor_scale_workspace_bytes(int64_t n, int x_dtype);
int nvfp4_tensor_scale(const void* x, int x_dtype, int64_t n, float* scale, void* workspace, size_t workspace_bytes,
                       mxf_stream stream);

/*
 * fp4_quantize - a matrix to 4-bit blocks, along its rows, its columns, or both from one read:
 *   MXFP4 (fmt MXF_W_MXFP4): blocks of B = 32, scale 2^(byte - 127) as in mxfp4_quantize_act, d = scale
 *   NVFP4 (MXF_W_NVFP4): blocks of B = 16, scale s = E4M3(amax / (6 g)) (round to nearest even,
 *     at most 448), d = s g; a block whose d is below 2^-126 is stored as zeros
 *   code = E2M1(x / d) in fp32, the sign kept, at most 6: to nearest, ties to even, or with rnd the
 *     upper of the two neighbours of |x / d| where the part above the lower one, as a share of
 *     their distance, exceeds (rnd + 1/2) / 256
 *   x            [rows][cols] fp32 or bf16 (x_dtype)
 *   tensor_scale [1] fp32 on the device (4-byte aligned), positive: g (NULL: 1; MXFP4 has none)
 *   rnd          [rows][cols] random bytes, the same for both directions; NULL: to nearest
 *   q, q_scale   [rows][cols/2], [rows][cols/B] (both NULL: not wanted)
 *   qt, qt_scale the codes of x^T, blocks along x's columns: [cols][R/2], [cols][R/B] with R = rows
 *                rounded up to 128; elements past the rows are zeros (both NULL: not wanted)
 * These are the operands of fp4_gemm, which sums over K % 128 == 0: qt, qt_scale for any rows; q, q_scale where
 * cols % 128 == 0 (x's columns filled up with zeros before this call give that and add nothing). q, q_scale are
 * the weights of the calls above, too. MXFP4 along rows to nearest is mxfp4_quantize_act's MXF_E2M1, bit for bit.
 * Values that are not finite are not handled: they spoil their own block (and a tensor scale taken from them).
 * Requires cols % 32 == 0, cols < 2^22 and at most 2^23 tiles of 128 x 128 (transposed), or rows cols
 * below 2^36. rows == 0 is a no-op. Errors: NULL, SHAPE (a tensor scale with MXFP4, too), ALIGN, FORMAT,
 * UNSUPPORTED.
 */
int fp4_quantize(const void* x, int x_dtype, int64_t rows, int64_t cols, int fmt, const float* tensor_scale,
                 const uint8_t* rnd, uint8_t* q, uint8_t* q_scale, uint8_t* qt, uint8_t* qt_scale, mxf_stream stream);

/*
 * fp4_dequantize - out [rows][cols] (fp32 or bf16) = E2M1 value x block scale x g in fp32, rounded to
 * out_dtype (exact where g is a power of two and nothing leaves the type's range). Arguments
 * as fp4_quantize writes them along the rows; a transposed result is read with its own rows and cols.
 * Requires cols % 32 == 0. rows == 0 is a no-op. Errors: NULL, SHAPE, ALIGN, FORMAT, UNSUPPORTED.
 */
int fp4_dequantize(const uint8_t* q, const uint8_t* q_scale, int64_t rows, int64_t cols, int fmt,
                   const float* tensor_scale, void* out, int out_dtype, mxf_stream stream);

/*
 * fp4_gemm - the product of two quantised matrices, C = g_a g_b A_hat * B_hat^T
 *   a, a_scale   [M][K/2] E2M1 codes, [M][K/32] UE8M0 bytes (fmt MXF_W_MXFP4) or [M][K/16] UE4M3 bytes
 *                (MXF_W_NVFP4), as fp4_quantize writes them;  b, b_scale  [N][K/2], [N][K/32] or [N][K/16]
 *   a_tensor_scale, b_tensor_scale  [1] fp32 on the device (4-byte aligned): g_a, g_b of NVFP4 (NULL: 1;
 *                MXFP4 has none)
 *   c            [M][N] fp32 or bf16 (c_dtype): the fp32 sum times g_a g_b in fp32, rounded to c_dtype. The
 *                scales' exponents are applied together, so that neither alone can overflow or underflow
 *   workspace    fp4_gemm_workspace_bytes(M, N, K, fmt) bytes (0: none needed, may be NULL), 16-byte
 *                aligned, contents irrelevant: K slices' sums, added in a fixed order; calls that may
 *                overlap need one each
 * A linear layer y = x W^T of [T][I] by [O][I] (I and O multiples of 128, or x, W and dy filled up with columns
 * of zeros before they are quantised) and its gradients: y = fp4_gemm(q(x), q(W)), dx =
 * fp4_gemm(q(dy), qt(W)), dW = fp4_gemm(qt(dy), qt(x)), q and qt as fp4_quantize's.
 * Every product is exact (NVFP4: code x scale is exact in the fp16 operands), accumulation in fp32.
 * Requires K % 128 == 0, N % 16 == 0, K < 2^24, M N < 2^34 and at most 2^21 tiles of 128 x 128. The
 * UE8M0 byte 255 and the UE4M3 byte 0x7F (NaN) are not valid scales. M == 0 is a no-op; K == 0 is refused
 * (SHAPE): the weight gradient of no tokens is zeros, which the caller writes.
 * Errors: NULL, SHAPE (a tensor scale with MXFP4, too), ALIGN, FORMAT, UNSUPPORTED, WORKSPACE.
 */
size_t fp4_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int fmt);
int fp4_gemm(const uint8_t* a, const uint8_t* a_scale, int64_t M, const uint8_t* b, const uint8_t* b_scale, int64_t N,
             int64_t K, int fmt, const float* a_tensor_scale, const float* b_tensor_scale, void* c, int c_dtype,
             void* workspace, size_t workspace_bytes, mxf_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4_MOE_H */
