// block_abi.cu -- the extern "C" entry points declared in include/moe_block.h: argument checks on the host
// (a status, nothing launched on failure), then the launches of the kernel files.
#include <climits>
#include <cmath>
#include <cstdint>

#include "block_launch.h"
#include "moe_block.h"
#include "moe_host.h"

using moe::aligned;
using moe::from_cuda;
using moe::make_ctx;

// The layout, and that columns fit: every offset into the buffers stays far inside int64.
static moe_status_t check_rows(moe_mode_t mode, int E, int M, int64_t* rows, int n, int k, const int64_t* seg,
                               const int32_t* count, const int32_t* status) {
    if (mode != MOE_MODE_NORMAL && mode != MOE_MODE_MASKED) return MOE_ERR_INVALID_ARG;
    if (E < 1) return MOE_ERR_INVALID_ARG;
    if (E > MOE_MAX_EXPERTS) return MOE_ERR_UNSUPPORTED;
    const bool masked = mode == MOE_MODE_MASKED;
    if (masked) {
        if (M < 1) return MOE_ERR_INVALID_ARG;
        *rows = int64_t(E) * M;
    }
    if (*rows < 0 || n <= 0 || n % 8 != 0 || k <= 0 || k % 8 != 0) return MOE_ERR_INVALID_ARG;
    if (*rows > INT32_MAX || n > (1 << 24) || k > (1 << 24)) return MOE_ERR_UNSUPPORTED;
    if (!status || !count || (!masked && !seg)) return MOE_ERR_INVALID_ARG;
    if (!aligned(seg, 8) || !aligned(count, 4) || !aligned(status, 4)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

static moe_status_t row_gemm(moe_mode_t mode, moe::RowOp op, bool kn, const uint16_t* a, int E, int M, int64_t rows,
                             int n, int k, const int64_t* seg, const int32_t* count, const uint16_t* w, uint16_t* out,
                             uint16_t* gate_up, int32_t* status, moe_stream_t stream) {
    moe_status_t st = check_rows(mode, E, M, &rows, n, k, seg, count, status);
    if (st != MOE_OK) return st;
    if ((rows / 256 + E) * (int64_t(n) / 128 + 1) > INT32_MAX / 2) return MOE_ERR_UNSUPPORTED;  // tiles
    if (op == moe::RowOp::kSwiglu && n > (1 << 23)) return MOE_ERR_UNSUPPORTED;
    if (rows == 0) return MOE_OK;
    if (!a || !w || !out || (op == moe::RowOp::kDswiglu && !gate_up)) return MOE_ERR_INVALID_ARG;
    if (!aligned(a, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(gate_up, 16)) return MOE_ERR_INVALID_ARG;
    moe::LaunchCtx ctx;
    st = make_ctx(stream, &ctx);
    if (st != MOE_OK) return st;
    const moe::RowLayout layout{E, mode == MOE_MODE_MASKED ? M : 0, rows, seg, count, status};
    return from_cuda(moe::launch_row_gemm(ctx, moe::RowGemm{layout, op, kn, a, n, k, w, out, gate_up}));
}

extern "C" {

moe_status_t moe_expert_gemm_bf16(moe_mode_t mode, const uint16_t* a, int num_experts, int max_tokens_per_expert,
                                  int64_t rows, int n, int k, const int64_t* seg_indptr, const int32_t* masked_m,
                                  moe_weights_t weights, const uint16_t* w, uint16_t* out, int32_t* dev_status,
                                  moe_stream_t stream) {
    if (weights != MOE_WEIGHTS_NK && weights != MOE_WEIGHTS_KN) return MOE_ERR_INVALID_ARG;
    return row_gemm(mode, moe::RowOp::kPlain, weights == MOE_WEIGHTS_KN, a, num_experts, max_tokens_per_expert, rows, n,
                    k, seg_indptr, masked_m, w, out, nullptr, dev_status, stream);
}

moe_status_t moe_expert_gemm_swiglu_bf16(moe_mode_t mode, const uint16_t* a, int num_experts,
                                         int max_tokens_per_expert, int64_t rows, int inter, int k,
                                         const int64_t* seg_indptr, const int32_t* masked_m, const uint16_t* w13,
                                         uint16_t* h, uint16_t* gate_up, int32_t* dev_status, moe_stream_t stream) {
    return row_gemm(mode, moe::RowOp::kSwiglu, false, a, num_experts, max_tokens_per_expert, rows, inter, k, seg_indptr,
                    masked_m, w13, h, gate_up, dev_status, stream);
}

moe_status_t moe_expert_gemm_dswiglu_bf16(moe_mode_t mode, const uint16_t* grad_out, int num_experts,
                                          int max_tokens_per_expert, int64_t rows, int inter, int k,
                                          const int64_t* seg_indptr, const int32_t* masked_m, const uint16_t* w2,
                                          const uint16_t* gate_up, uint16_t* grad_gate_up, int32_t* dev_status,
                                          moe_stream_t stream) {
    return row_gemm(mode, moe::RowOp::kDswiglu, true, grad_out, num_experts, max_tokens_per_expert, rows, inter, k,
                    seg_indptr, masked_m, w2, grad_gate_up, const_cast<uint16_t*>(gate_up), dev_status, stream);
}

moe_status_t moe_expert_wgrad_bf16(moe_mode_t mode, const uint16_t* a, const uint16_t* b, int num_experts,
                                   int max_tokens_per_expert, int64_t rows, int m, int n, const int64_t* seg_indptr,
                                   const int32_t* masked_m, moe_grad_t grad, int accumulate, void* out,
                                   int32_t* dev_status, moe_stream_t stream) {
    if (grad != MOE_GRAD_BF16 && grad != MOE_GRAD_FP32) return MOE_ERR_INVALID_ARG;
    if (accumulate != 0 && accumulate != 1) return MOE_ERR_INVALID_ARG;
    moe_status_t st = check_rows(mode, num_experts, max_tokens_per_expert, &rows, m, n, seg_indptr, masked_m, dev_status);
    if (st != MOE_OK) return st;
    if (int64_t(num_experts) * (m / 256 + 1) * (n / 256 + 1) > INT32_MAX / 2) return MOE_ERR_UNSUPPORTED;  // tiles
    if ((mode == MOE_MODE_MASKED ? max_tokens_per_expert : rows) > moe::kMostSummedRows) return MOE_ERR_UNSUPPORTED;
    if (!out || !aligned(out, 16)) return MOE_ERR_INVALID_ARG;
    if (rows > 0 && (!a || !b)) return MOE_ERR_INVALID_ARG;
    if (!aligned(a, 16) || !aligned(b, 16)) return MOE_ERR_INVALID_ARG;
    moe::LaunchCtx ctx;
    st = make_ctx(stream, &ctx);
    if (st != MOE_OK) return st;
    const moe::RowLayout layout{num_experts, mode == MOE_MODE_MASKED ? max_tokens_per_expert : 0, rows, seg_indptr,
                                masked_m, dev_status};
    return from_cuda(moe::launch_weight_grad(
        ctx, moe::WeightGrad{layout, a, b, m, n, grad == MOE_GRAD_FP32, accumulate != 0, out}));
}

moe_status_t moe_combine_backward(moe_mode_t mode, const uint16_t* grad_out, const uint16_t* expert_out,
                                  int64_t num_tokens, int hidden, int topk, int num_experts,
                                  int max_tokens_per_expert, int64_t expert_out_rows, const int32_t* topk_ids,
                                  const int32_t* src2dst, const int64_t* seg_indptr, const float* topk_weights,
                                  uint16_t* grad_expert_out, float* grad_topk_weights, int32_t* dev_status,
                                  moe_stream_t stream) {
    if (mode != MOE_MODE_NORMAL && mode != MOE_MODE_MASKED) return MOE_ERR_INVALID_ARG;
    moe_status_t st = moe::check_shape(num_tokens, topk, num_experts);
    if (st != MOE_OK) return st;
    if (hidden <= 0 || hidden % 8 != 0) return MOE_ERR_INVALID_ARG;
    const bool masked = mode == MOE_MODE_MASKED;
    if (masked && max_tokens_per_expert < 1) return MOE_ERR_INVALID_ARG;
    if (!masked && (expert_out_rows < 0 || (expert_out_rows != 0 && expert_out_rows < num_tokens * topk)))
        return MOE_ERR_INVALID_ARG;
    if (!dev_status || !aligned(dev_status, 4)) return MOE_ERR_INVALID_ARG;
    if (!grad_expert_out && !grad_topk_weights) return MOE_ERR_INVALID_ARG;
    if (num_tokens == 0) return MOE_OK;
    if (!grad_out || !src2dst || (grad_expert_out && !topk_weights) || (grad_topk_weights && !expert_out))
        return MOE_ERR_INVALID_ARG;
    if (masked && (!topk_ids || !seg_indptr)) return MOE_ERR_INVALID_ARG;
    if (!aligned(grad_out, 16) || !aligned(expert_out, 16) || !aligned(grad_expert_out, 16) || !aligned(topk_ids, 4) ||
        !aligned(src2dst, 4) || !aligned(seg_indptr, 8) || !aligned(topk_weights, 4) || !aligned(grad_topk_weights, 4))
        return MOE_ERR_INVALID_ARG;
    moe::LaunchCtx ctx;
    st = make_ctx(stream, &ctx);
    if (st != MOE_OK) return st;
    return from_cuda(moe::launch_combine_backward(
        ctx, moe::CombineGrad{masked, grad_out, grad_topk_weights ? expert_out : nullptr, num_tokens, hidden, topk,
                              num_experts, max_tokens_per_expert,
                              expert_out_rows > 0 ? expert_out_rows : num_tokens * topk, topk_ids, src2dst, seg_indptr,
                              topk_weights, grad_expert_out, grad_topk_weights, dev_status}));
}

static moe_status_t check_norm_shape(int64_t T, int H) {
    if (T < 0 || H <= 0 || H % 8 != 0) return MOE_ERR_INVALID_ARG;
    if (T > INT32_MAX || H > MOE_NORM_MAX_HIDDEN) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

moe_status_t moe_rmsnorm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, float eps,
                         int64_t num_tokens, int hidden, moe_quant_t quant, uint16_t* out, uint8_t* codes,
                         void* scales, uint16_t* sum, float* rstd, moe_stream_t stream) {
    if (quant != MOE_QUANT_NONE && quant != MOE_QUANT_FP8_G128 && quant != MOE_QUANT_FP8_G128_UE8M0)
        return MOE_ERR_INVALID_ARG;
    moe_status_t st = check_norm_shape(num_tokens, hidden);
    if (st != MOE_OK) return st;
    const bool fp8 = quant != MOE_QUANT_NONE;
    if (fp8 && hidden % 128 != 0) return MOE_ERR_INVALID_ARG;
    if (!(eps > 0.0f) || !std::isfinite(eps)) return MOE_ERR_INVALID_ARG;
    if (num_tokens == 0) return MOE_OK;
    if (!x || !weight || (fp8 ? !codes || !scales : !out)) return MOE_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(out, 16) || !aligned(codes, 16) ||
        !aligned(sum, 16) || !aligned(rstd, 4) || (quant == MOE_QUANT_FP8_G128 && !aligned(scales, 4)))
        return MOE_ERR_INVALID_ARG;
    moe::LaunchCtx ctx;
    st = make_ctx(stream, &ctx);
    if (st != MOE_OK) return st;
    return from_cuda(moe::launch_rmsnorm(ctx, moe::Norm{x, residual, weight, eps, num_tokens, hidden, int(quant), out,
                                                        codes, scales, residual ? sum : nullptr, rstd}));
}

size_t moe_rmsnorm_backward_workspace_size(int64_t num_tokens, int hidden) {
    if (check_norm_shape(num_tokens, hidden) != MOE_OK) return 0;
    return size_t(moe::norm_backward_blocks(num_tokens, hidden)) * size_t(hidden) * sizeof(float);
}

moe_status_t moe_rmsnorm_backward(const uint16_t* grad_out, const uint16_t* s, const uint16_t* weight,
                                  const float* rstd, const uint16_t* grad_sum, int64_t num_tokens, int hidden,
                                  uint16_t* grad_x, float* grad_weight, void* workspace, size_t workspace_bytes,
                                  moe_stream_t stream) {
    moe_status_t st = check_norm_shape(num_tokens, hidden);
    if (st != MOE_OK) return st;
    if (!grad_weight || !aligned(grad_weight, 16)) return MOE_ERR_INVALID_ARG;
    if (num_tokens > 0) {
        if (!grad_out || !s || !weight || !rstd || !grad_x || !workspace) return MOE_ERR_INVALID_ARG;
        if (!aligned(grad_out, 16) || !aligned(s, 16) || !aligned(weight, 16) || !aligned(rstd, 4) ||
            !aligned(grad_sum, 16) || !aligned(grad_x, 16) || !aligned(workspace, 16))
            return MOE_ERR_INVALID_ARG;
        if (workspace_bytes < moe_rmsnorm_backward_workspace_size(num_tokens, hidden)) return MOE_ERR_INVALID_ARG;
    }
    moe::LaunchCtx ctx;
    st = make_ctx(stream, &ctx);
    if (st != MOE_OK) return st;
    return from_cuda(moe::launch_rmsnorm_backward(ctx, moe::NormGrad{grad_out, s, weight, rstd, grad_sum, num_tokens,
                                                                     hidden, grad_x, grad_weight,
                                                                     static_cast<float*>(workspace)}));
}

}  // extern "C"
