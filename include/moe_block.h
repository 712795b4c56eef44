/*
 * moe_block.h -- C ABI of a MoE block's operators in bf16, for training and for serving bf16 weights.
 *
 *   moe_expert_gemm_bf16           rows of a dispatched layout x their expert's weights; with transposed
 *                                  weights the gradient with respect to the rows
 *   moe_expert_gemm_swiglu_bf16    the gate and up products with SwiGLU
 *   moe_expert_gemm_dswiglu_bf16   the down product's gradient through SwiGLU
 *   moe_expert_wgrad_bf16          the gradient with respect to the weights: a sum over each expert's rows
 *   moe_combine_backward           the gradient of moe_combine(_ex)
 *   moe_rmsnorm                    root-mean-square norm of x + residual: bf16 rows, and FP8 rows with the
 *                                  dispatch's scales
 *   moe_rmsnorm_backward           its gradient
 *
 * The products read what moe_dispatch(_ex) with MOE_QUANT_NONE writes, in the contiguous and the masked
 * layout. The gradient of that dispatch is moe_combine_ex with weights of 1. The dispatcher pages show
 * neither the experts nor gradients: these calls have no counterpart on them, but for the FP8 rows, which
 * are those of sglang_per_token_group_quant_fp8 ("sglang token_dispatcher/deepep.py" page,
 * _DeepEPDispatcherImplNormal.dispatch_a).
 *
 * Conventions (device pointers, stream order, no allocation, status codes, first error wins in
 * *dev_status) are those of moe_dispatch.h. Sums are fp32; a bf16 result is rounded once.
 */
#ifndef MOE_BLOCK_H
#define MOE_BLOCK_H

#include "moe_dispatch.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How the weights of a product lie in memory. */
typedef enum {
    MOE_WEIGHTS_NK = 0,  /* w [E, n, k]: out[r, j] = sum_k a[r, k] * w[e, j, k]                               */
    MOE_WEIGHTS_KN = 1   /* w [E, k, n]: out[r, j] = sum_k a[r, k] * w[e, k, j], the gradient with respect to
                            the rows of a product whose weights are [E, k, n] in MOE_WEIGHTS_NK             */
} moe_weights_t;

typedef enum { MOE_GRAD_BF16 = 0, MOE_GRAD_FP32 = 1 } moe_grad_t;

#define MOE_NORM_MAX_HIDDEN 32768

/*
 * moe_expert_gemm_bf16 -- out[r, j] = bf16_rn(sum_k a[r, k] * w(e, j, k)) for every row r of every expert e.
 *   The rows of expert e:  masked:  e*M + [0, masked_m[e])
 *                          normal:  seg_indptr[e] + [0, masked_m[e])
 *   as moe_route_meta(_ex) and moe_dispatch(_ex) leave them (aligned segments or not). Other rows of out
 *   are not written, and what other rows of `a` hold does not matter (NaNs neither).
 *   A count above M (masked) or rows beyond `rows` (normal) are cut off and reported as MOE_ERR_CAPACITY; a
 *   negative count or start is skipped and reported as MOE_ERR_INVALID_ARG. No row belongs to two experts:
 *   segments that overlap so far that they have more than rows / 256 + E tiles of 256 rows are reported as
 *   MOE_ERR_INVALID_ARG, and nothing is written.
 * Arguments:
 *   num_experts (E)  1..MOE_MAX_EXPERTS.
 *   max_tokens_per_expert (M)  masked: >= 1. Ignored in normal mode.
 *   rows             normal: rows of `a` and `out` (their capacity). Ignored in masked mode (E*M).
 *                    At most INT32_MAX rows in either mode.
 *   n, k             columns of out, and of a: multiples of 8, at most 2^24.
 *   seg_indptr       [E+1] int64 (normal; may be NULL in masked mode).
 *   masked_m         [E] int32: the pairs of each expert.
 *   a [rows, k], w, out [rows, n]  bf16, 16-byte aligned; out overlaps neither a nor w.
 * Returns MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED or MOE_ERR_CUDA.
 */
moe_status_t moe_expert_gemm_bf16(moe_mode_t mode, const uint16_t *a, int num_experts, int max_tokens_per_expert,
                                  int64_t rows, int n, int k, const int64_t *seg_indptr, const int32_t *masked_m,
                                  moe_weights_t weights, const uint16_t *w, uint16_t *out, int32_t *dev_status,
                                  moe_stream_t stream);

/*
 * moe_expert_gemm_swiglu_bf16 -- for the same rows, with w13[e] the `inter` gate rows followed by the `inter`
 * up rows of expert e (MOE_WEIGHTS_NK):
 *   G = sum_k a[r, k] * w13[e, i, k],  U = sum_k a[r, k] * w13[e, inter + i, k]
 *   h[r, i] = bf16_rn(U * (G / (1 + exp(-G)))), from the fp32 sums
 *   gate_up[r, i] = bf16_rn(G), gate_up[r, inter + i] = bf16_rn(U), if gate_up is not NULL: what
 *   moe_expert_gemm_dswiglu_bf16 needs.
 *   w13 [E, 2*inter, k], h [rows, inter], gate_up [rows, 2*inter], inter a multiple of 8; else as above.
 */
moe_status_t moe_expert_gemm_swiglu_bf16(moe_mode_t mode, const uint16_t *a, int num_experts,
                                         int max_tokens_per_expert, int64_t rows, int inter, int k,
                                         const int64_t *seg_indptr, const int32_t *masked_m, const uint16_t *w13,
                                         uint16_t *h, uint16_t *gate_up, int32_t *dev_status, moe_stream_t stream);

/*
 * moe_expert_gemm_dswiglu_bf16 -- the gradient of out = h w2[e]^T, h = U * silu(G), with respect to G and U:
 *   dh = sum_k grad_out[r, k] * w2[e, k, i],  p = 1 / (1 + exp(-G))
 *   grad_gate_up[r, i] = bf16_rn(dh * U * p * (1 + G * (1 - p)))
 *   grad_gate_up[r, inter + i] = bf16_rn(dh * G * p)
 * with G, U = gate_up[r, i], gate_up[r, inter + i], and dh in fp32. The gradients are rounded to bf16 because
 * the products that read them (moe_expert_gemm_bf16 with MOE_WEIGHTS_KN, moe_expert_wgrad_bf16) take bf16 rows:
 * the rows' gradient through both is 0.0023 off in norm, and would be 0.0017 off, its own rounding, if they were
 * kept in fp32. p and 1 - p are within 2^-20 (for G below -87 the step of a subnormal exp(G) comes on top). The
 * gradients of an infinite or NaN G or U are unspecified.
 *   grad_out [rows, k], w2 [E, k, inter], gate_up and grad_gate_up [rows, 2*inter]; grad_gate_up may be gate_up
 *   itself, and overlaps it in no other way; else as above.
 */
moe_status_t moe_expert_gemm_dswiglu_bf16(moe_mode_t mode, const uint16_t *grad_out, int num_experts,
                                          int max_tokens_per_expert, int64_t rows, int inter, int k,
                                          const int64_t *seg_indptr, const int32_t *masked_m, const uint16_t *w2,
                                          const uint16_t *gate_up, uint16_t *grad_gate_up, int32_t *dev_status,
                                          moe_stream_t stream);

/*
 * moe_expert_wgrad_bf16 -- out[e, i, j] (+)= sum over the rows r of expert e of a[r, i] * b[r, j]: with the
 * gradient of a product's results as `a` and its rows as `b`, the gradient of its weights in MOE_WEIGHTS_NK.
 *   An expert without rows gets zeros (accumulate: keeps what it has). What rows outside the experts' counts
 *   hold does not matter. Segments may overlap. fp32 sums in an order that depends on the arguments alone; they are the
 *   tensor core's, which cuts where an addition would round: 4.8e-7 off in norm over 512 rows (1.6e-7 rounded).
 *   m, n             columns of a and of b: multiples of 8, at most 2^24
 *   rows             (masked: max_tokens_per_expert) at most 2^26 here
 *   grad             type of out: MOE_GRAD_BF16 (rounded once) or MOE_GRAD_FP32
 *   accumulate       0: out is overwritten; 1: the sum is added to it in fp32 (MOE_GRAD_BF16: and rounded)
 *   a [rows, m], b [rows, n] bf16; out [E, m, n]; all 16-byte aligned, out overlaps neither; else as above.
 */
moe_status_t moe_expert_wgrad_bf16(moe_mode_t mode, const uint16_t *a, const uint16_t *b, int num_experts,
                                   int max_tokens_per_expert, int64_t rows, int m, int n, const int64_t *seg_indptr,
                                   const int32_t *masked_m, moe_grad_t grad, int accumulate, void *out,
                                   int32_t *dev_status, moe_stream_t stream);

/*
 * moe_combine_backward -- the gradient of moe_combine_ex's out with respect to its rows and weights:
 *   grad_expert_out[row(t, k), :] = bf16_rn(topk_weights[t, k] * grad_out[t, :])
 *   grad_topk_weights[t, k] = sum_h grad_out[t, h] * expert_out[row(t, k), h], 0 for a slot without a row
 *   with row(t, k) as moe_combine_ex has it. Other rows of grad_expert_out are not written. Either output may
 *   be NULL (grad_topk_weights NULL: expert_out is not read and may be NULL). grad_expert_out may be
 *   expert_out itself, and overlaps it in no other way.
 *   grad_out [T, hidden], hidden a multiple of 8; topk_ids, seg_indptr: masked mode; expert_out_rows as for
 *   moe_combine_ex, of both row buffers. Errors that the rows show are reported as there.
 */
moe_status_t moe_combine_backward(moe_mode_t mode, const uint16_t *grad_out, const uint16_t *expert_out,
                                  int64_t num_tokens, int hidden, int topk, int num_experts,
                                  int max_tokens_per_expert, int64_t expert_out_rows, const int32_t *topk_ids,
                                  const int32_t *src2dst, const int64_t *seg_indptr, const float *topk_weights,
                                  uint16_t *grad_expert_out, float *grad_topk_weights, int32_t *dev_status,
                                  moe_stream_t stream);

/*
 * moe_rmsnorm -- for every row t:
 *   s = bf16_rn(x[t] + residual[t])  (x[t] without a residual), r = 1 / sqrt(mean(s^2) + eps)
 *   y = (s * r) * weight             in fp32
 *   out[t]    = bf16_rn(y)                                                  (out not NULL)
 *   codes[t], scales[t] = y quantised as moe_dispatch does for MOE_QUANT_FP8_G128 or
 *                         MOE_QUANT_FP8_G128_UE8M0, from the unrounded y    (quant not MOE_QUANT_NONE)
 *   sum[t]    = s (only with a residual)                                    (sum not NULL)
 *   rstd[t]   = r                                                           (rstd not NULL)
 *   hidden           a multiple of 8 (of 128 with FP8), at most MOE_NORM_MAX_HIDDEN
 *   x, residual, out, sum [T, hidden] bf16, weight [hidden] bf16, codes [T, hidden]: 16-byte aligned.
 *                    scales [T, hidden/128] fp32 or UE8M0 bytes. rstd [T] fp32. out, codes or both.
 *                    sum may be x or residual itself; no other output overlaps an input.
 *   eps              > 0 and finite
 * All in binary32: a row whose squares overflow it (values beyond 2^63) has r = 0. A row of infinities or NaNs
 * leaves the others as they are.
 */
moe_status_t moe_rmsnorm(const uint16_t *x, const uint16_t *residual, const uint16_t *weight, float eps,
                         int64_t num_tokens, int hidden, moe_quant_t quant, uint16_t *out, uint8_t *codes,
                         void *scales, uint16_t *sum, float *rstd, moe_stream_t stream);

/* Bytes of workspace that moe_rmsnorm_backward needs (any contents, 16-byte aligned); 0 for arguments it would
 * reject or that need none. Calls that share a workspace must not overlap on the GPU. */
size_t moe_rmsnorm_backward_workspace_size(int64_t num_tokens, int hidden);

/*
 * moe_rmsnorm_backward -- with s and r of moe_rmsnorm (sum, or x without a residual; rstd), g = grad_out:
 *   grad_x[t]   = bf16_rn(r * (g * weight - (s * r) * mean(g * weight * (s * r))) + grad_sum[t]): the gradient
 *                 of x and of the residual alike; grad_sum [T, hidden] (NULL: 0) is what else flows into s
 *   grad_weight = sum_t g[t] * (s[t] * r[t])      [hidden] fp32, in an order that depends on T and hidden alone
 *                 on a given GPU; zeros without tokens
 *   All rows bf16, 16-byte aligned. grad_x may be grad_out or grad_sum itself.
 */
moe_status_t moe_rmsnorm_backward(const uint16_t *grad_out, const uint16_t *s, const uint16_t *weight,
                                  const float *rstd, const uint16_t *grad_sum, int64_t num_tokens, int hidden,
                                  uint16_t *grad_x, float *grad_weight, void *workspace, size_t workspace_bytes,
                                  moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_H */
