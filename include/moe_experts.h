/*
 * moe_experts.h -- C ABI of the expert operators between moe_dispatch and moe_combine.
 *
 *   moe_quantize_nvfp4       bf16 rows -> e2m1 codes + e4m3 block scales (weights, activations)
 *   moe_dequantize_nvfp4     the reverse
 *   moe_expert_gemm          rows of a dispatched layout x their expert's weights -> bf16
 *   moe_expert_gemm_swiglu   the gate and up products, SwiGLU and requantisation in one kernel:
 *                            its output is the input of the down product (moe_expert_gemm)
 *   moe_layer_few_tokens     a whole layer (experts and weighted sum) for up to
 *                            MOE_LAYER_MAX_TOKENS tokens in two kernels, without a dispatch
 *
 * The dispatcher pages stop at the experts: FlashinferDispatcher.dispatch ("sglang
 * token_dispatcher/flashinfer.py" page) hands NVFP4 codes and interleaved block scales, and
 * low_latency_dispatch ("sglang token_dispatcher/deepep.py" page) a masked layout, to a MoE GEMM
 * that they do not show. These calls are that consumer for NVFP4 rows in the contiguous and masked
 * layouts of moe_dispatch(_ex); the one-row-per-partition layout of moe_dispatch_partitioned(_ex)
 * is not read by them. They have no counterpart on the pages.
 *
 * Conventions (device pointers, stream order, no allocation, status codes, first error wins in
 * *dev_status) are those of moe_dispatch.h. NVFP4 matrices hold value(code) * value(scale): codes
 * e2m1, two per byte (even element in the low nibble), one e4m3 scale per 16 consecutive elements
 * of a row, in one of the layouts of moe_scale_layout_t (MOE_SCALES_COL_MAJOR is FP8 only).
 */
#ifndef MOE_EXPERTS_H
#define MOE_EXPERTS_H

#include "moe_dispatch.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_LAYER_MAX_TOKENS 64   /* T of moe_layer_few_tokens */

/*
 * moe_quantize_nvfp4 -- quantise `groups` matrices [rows, hidden] of bf16, each with its own
 * global scale g, per block of 16 consecutive elements, in binary32 with round to nearest even, in
 * the order written:
 *   sf = e4m3_rn_satfinite((amax / 6) * g),  q = e2m1_rn_satfinite(x * (g / sf)), 0 if sf is 0:
 * the codes and scales of moe_dispatch's MOE_QUANT_NVFP4_B16. The usual g is 448 * 6 / max|x| of
 * the matrix.
 *   x              [groups, rows, hidden] bf16, 16-byte aligned
 *   hidden         > 0, % 16 == 0; % 64 == 0 for MOE_SCALES_SWIZZLED_128X4
 *   global_scales  [groups] fp32
 *   codes          [groups, rows, hidden/2] out, 8-byte aligned
 *   scales         MOE_SCALES_ROW_MAJOR: [groups, rows, hidden/16] out; MOE_SCALES_SWIZZLED_128X4:
 *                  per group the tiles of its own [roundup(rows, 128), hidden/16] matrix, padding
 *                  rows zero, 4-byte aligned
 * Infinities and NaNs in x give unspecified codes in their own block only.
 * Returns MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED or MOE_ERR_CUDA.
 */
moe_status_t moe_quantize_nvfp4(const uint16_t *x, int64_t groups, int64_t rows, int hidden,
                                const float *global_scales, moe_scale_layout_t scale_layout, uint8_t *codes,
                                uint8_t *scales, moe_stream_t stream);

/*
 * moe_dequantize_nvfp4 -- out = bf16_rn((value(code) * value(scale)) / g): the product is exact in
 * binary32, the division rounds once to binary32. Arguments as moe_quantize_nvfp4; out
 * [groups, rows, hidden] bf16, 16-byte aligned.
 */
moe_status_t moe_dequantize_nvfp4(const uint8_t *codes, const uint8_t *scales, int64_t groups, int64_t rows,
                                  int hidden, const float *global_scales, moe_scale_layout_t scale_layout,
                                  uint16_t *out, moe_stream_t stream);

/*
 * moe_expert_gemm -- out[r, n] = bf16_rn(alpha[e] * sum_k a[r, k] * w[e, n, k]) for every row r of
 * every expert e; fp32 accumulation.
 *   The rows of expert e:  masked:  e*M + [0, masked_m[e])
 *                          normal:  seg_indptr[e] + [0, masked_m[e])
 *   as moe_route_meta(_ex) and moe_dispatch(_ex) leave them (aligned segments or not). Other rows
 *   of out are not written, and what other rows of `a` hold does not matter.
 *   A count above M (masked) or rows beyond `rows` (normal) are cut off and reported as
 *   MOE_ERR_CAPACITY; a negative count or start is skipped and reported as MOE_ERR_INVALID_ARG.
 *   No row belongs to two experts: segments that overlap so far that they have more than
 *   rows / 128 + E tiles of 128 rows are reported as MOE_ERR_INVALID_ARG, and nothing is written.
 * Arguments:
 *   num_experts (E)  1..MOE_MAX_EXPERTS.
 *   max_tokens_per_expert (M)  masked: >= 1. Ignored in normal mode.
 *   rows             normal: rows of `a` and `out` (their capacity). Ignored in masked mode (E*M).
 *                    At most INT32_MAX rows in either mode.
 *   n, k             columns of out, and of a and w: n % 16 == 0, k % 64 == 0.
 *   seg_indptr       [E+1] int64 (normal; may be NULL in masked mode).
 *   masked_m         [E] int32: the pairs of each expert.
 *   a_codes          [rows, k/2], 16-byte aligned. a_scales: one [rows, k/16] matrix over all rows,
 *                    MOE_SCALES_ROW_MAJOR or MOE_SCALES_SWIZZLED_128X4 (4-byte aligned).
 *   w_codes          [E, n, k/2], 16-byte aligned. w_scales: per expert the 128 x 4 tiles of its
 *                    [roundup(n, 128), k/16] matrix, 16-byte aligned (moe_quantize_nvfp4 with one
 *                    group per expert).
 *   alpha            [E] fp32, or NULL for 1: usually 1 / (g of the activations * g of the weights).
 *   out              [rows, n] bf16, 16-byte aligned.
 * Returns MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED or MOE_ERR_CUDA.
 */
moe_status_t moe_expert_gemm(moe_mode_t mode, const uint8_t *a_codes, const uint8_t *a_scales,
                             moe_scale_layout_t scale_layout, int num_experts, int max_tokens_per_expert,
                             int64_t rows, int n, int k, const int64_t *seg_indptr, const int32_t *masked_m,
                             const uint8_t *w_codes, const uint8_t *w_scales, const float *alpha, uint16_t *out,
                             int32_t *dev_status, moe_stream_t stream);

/*
 * moe_expert_gemm_swiglu -- for the same rows, with w13[e] the `inter` gate rows followed by the
 * `inter` up rows of expert e:
 *   G = alpha[e] * sum_k a[r, k] * w13[e, i, k],  U = alpha[e] * sum_k a[r, k] * w13[e, inter + i, k]
 *   h[r, i] = U * (G / (1 + exp(-G)))        in fp32, then quantised as moe_quantize_nvfp4 does
 *   with g = out_global_scale. The product's sums and exp are fp32 with their own rounding (h is
 *   within 2^-20 of its value for the G and U that the sums give; within 2^-19 for G below -87, where
 *   the step of a subnormal exp(G) comes on top), so a code next to a rounding boundary may differ
 *   from another evaluation's.
 * Arguments as moe_expert_gemm, with inter % 64 == 0 and
 *   w13_codes        [E, 2*inter, k/2]; w13_scales: per expert and half the tiles of its own
 *                    [roundup(inter, 128), k/16] matrix (moe_quantize_nvfp4 with 2*E groups).
 *   out_codes        [rows, inter/2] out, 16-byte aligned; out_scales one [rows, inter/16] matrix
 *                    over all rows in `scale_layout` (the layout of a_scales), 4-byte aligned.
 *                    Scales of rows that no expert has are not written.
 */
moe_status_t moe_expert_gemm_swiglu(moe_mode_t mode, const uint8_t *a_codes, const uint8_t *a_scales,
                                    moe_scale_layout_t scale_layout, int num_experts, int max_tokens_per_expert,
                                    int64_t rows, int inter, int k, const int64_t *seg_indptr,
                                    const int32_t *masked_m, const uint8_t *w13_codes, const uint8_t *w13_scales,
                                    const float *alpha, float out_global_scale, uint8_t *out_codes,
                                    uint8_t *out_scales, int32_t *dev_status, moe_stream_t stream);

/*
 * Bytes of workspace that moe_layer_few_tokens needs (any contents, 256-byte aligned); 0 for
 * arguments it would reject. Calls that share a workspace must not overlap on the GPU.
 */
size_t moe_layer_workspace_size(int64_t num_tokens, int topk, int hidden, int inter, int num_experts);

/*
 * moe_layer_few_tokens -- the layer's experts and their weighted sum, straight from token rows:
 *   h(t, e) = silu(alpha13[e] * W13[e][:inter] x_t) * (alpha13[e] * W13[e][inter:] x_t)
 *   out[t]  = bf16_rn( sum_{k valid} topk_weights[t, k] * alpha2[e] * (W2[e] h(t, e)) ),  e = topk_ids[t, k]
 * Weights are NVFP4 or bf16; activations are not quantised (the chain of moe_expert_gemm_swiglu and
 * moe_expert_gemm quantises x and h to NVFP4). With bf16 weights x enters as it is and h as the sum
 * of two bf16 values. With NVFP4 weights each block of 16 of x and of h enters as the sum of five
 * NVFP4 blocks, which leaves at most 2^-12 of the block's largest magnitude, typically 2^-18. A row
 * of x (of h) in which the largest of some eight (sixteen) neighbours, not all 0, lies more than 11
 * binary orders below the row's largest enters as five more such blocks for each 13 orders, each
 * five leaving that much of what the five before left: it keeps the values beside an outlier, and
 * costs its experts a reading of their weights for each. fp32 sums in an order that depends on the
 * arguments alone. A token without a valid slot gets zeros; a slot that names an expert twice counts
 * twice. Ids outside [-1, E) are skipped and reported as MOE_ERR_BAD_EXPERT_ID.
 * A token with infinities or NaNs gets unspecified values and leaves the other tokens' as they are.
 * Arguments:
 *   x                [T, hidden] bf16, 16-byte aligned; 0 <= T <= MOE_LAYER_MAX_TOKENS.
 *   topk_ids, topk_weights  [T, K] int32 / fp32, 1 <= K <= MOE_MAX_TOPK.
 *   weight_quant     MOE_QUANT_NVFP4_B16: w13 [E, 2*inter, hidden/2] and w2 [E, hidden, inter/2] codes,
 *                    their scales and per-expert factors as for the two products above (alpha is
 *                    1 / g of the weights alone here; NULL: 1); hidden % 64 == 0, inter % 64 == 0.
 *                    MOE_QUANT_NONE: w13 [E, 2*inter, hidden] and w2 [E, hidden, inter] bf16; scales NULL,
 *                    alpha NULL or per-expert factors; hidden % 16 == 0, inter % 16 == 0.
 *                    Weights 16-byte aligned, scales 16-byte aligned.
 *   out              [T, hidden] bf16, 16-byte aligned, must not overlap x.
 *   workspace        moe_layer_workspace_size(...) bytes.
 * Returns MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED (T > MOE_LAYER_MAX_TOKENS) or MOE_ERR_CUDA.
 */
moe_status_t moe_layer_few_tokens(const uint16_t *x, int64_t num_tokens, int hidden, int inter,
                                  const int32_t *topk_ids, const float *topk_weights, int topk, int num_experts,
                                  moe_quant_t weight_quant, const void *w13, const uint8_t *w13_scales,
                                  const float *alpha13, const void *w2, const uint8_t *w2_scales,
                                  const float *alpha2, uint16_t *out, void *workspace, size_t workspace_bytes,
                                  int32_t *dev_status, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EXPERTS_H */
