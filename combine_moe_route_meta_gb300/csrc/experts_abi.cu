// experts_abi.cu -- the extern "C" entry points declared in include/moe_experts.h: argument checks
// on the host (a status, nothing launched on failure), then the launches of the kernel files.
#include <climits>
#include <cstdint>

#include "experts_launch.h"
#include "moe_experts.h"
#include "moe_host.h"

using moe::aligned;
using moe::from_cuda;
using moe::make_ctx;

static moe_status_t check_quant(int64_t groups, int64_t rows, int hidden, moe_scale_layout_t layout,
                                const void* values, const float* gs, const uint8_t* codes, const uint8_t* scales,
                                bool* empty) {
    if (layout != MOE_SCALES_ROW_MAJOR && layout != MOE_SCALES_SWIZZLED_128X4) return MOE_ERR_INVALID_ARG;
    if (groups < 0 || rows < 0 || hidden <= 0 || hidden % 16 != 0) return MOE_ERR_INVALID_ARG;
    if (layout == MOE_SCALES_SWIZZLED_128X4 && (hidden % 64 != 0 || !aligned(scales, 4))) return MOE_ERR_INVALID_ARG;
    // every offset (the padded rows' too) stays far inside int64
    if (groups > INT32_MAX || rows > INT32_MAX - 128 || (rows > 0 && groups > (int64_t(1) << 46) / hidden / (rows + 127)))
        return MOE_ERR_UNSUPPORTED;
    *empty = groups == 0 || rows == 0;
    if (*empty) return MOE_OK;
    if (!values || !gs || !codes || !scales) return MOE_ERR_INVALID_ARG;
    if (!aligned(values, 16) || !aligned(codes, 8) || !aligned(gs, 4)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

static moe_status_t check_gemm(moe_mode_t mode, moe_scale_layout_t layout, int E, int M, int64_t* rows, int n, int k,
                               const int64_t* seg, const int32_t* count, const uint8_t* a, const uint8_t* a_sf,
                               const uint8_t* w, const uint8_t* w_sf, const float* alpha, const int32_t* status) {
    if (mode != MOE_MODE_NORMAL && mode != MOE_MODE_MASKED) return MOE_ERR_INVALID_ARG;
    if (layout != MOE_SCALES_ROW_MAJOR && layout != MOE_SCALES_SWIZZLED_128X4) return MOE_ERR_INVALID_ARG;
    if (E < 1) return MOE_ERR_INVALID_ARG;
    if (E > MOE_MAX_EXPERTS) return MOE_ERR_UNSUPPORTED;
    const bool masked = mode == MOE_MODE_MASKED;
    if (masked) {
        if (M < 1) return MOE_ERR_INVALID_ARG;
        *rows = int64_t(E) * M;
    }
    if (*rows < 0 || n <= 0 || n % 16 != 0 || k <= 0 || k % 64 != 0) return MOE_ERR_INVALID_ARG;
    if (*rows > INT32_MAX || n > (1 << 24) || k > (1 << 24)) return MOE_ERR_UNSUPPORTED;
    if ((*rows / 128 + E) * (int64_t(n) / 128 + 1) > INT32_MAX / 2) return MOE_ERR_UNSUPPORTED;  // tiles
    if (!status || !count || (!masked && !seg)) return MOE_ERR_INVALID_ARG;
    if (*rows > 0 && (!a || !a_sf || !w || !w_sf)) return MOE_ERR_INVALID_ARG;
    if (!aligned(a, 16) || !aligned(a_sf, 4) || !aligned(w, 16) || !aligned(w_sf, 16) || !aligned(alpha, 4) ||
        !aligned(seg, 8) || !aligned(count, 4) || !aligned(status, 4))
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

extern "C" {

moe_status_t moe_quantize_nvfp4(const uint16_t* x, int64_t groups, int64_t rows, int hidden,
                                const float* global_scales, moe_scale_layout_t scale_layout, uint8_t* codes,
                                uint8_t* scales, moe_stream_t stream) {
    bool empty;
    moe_status_t st = check_quant(groups, rows, hidden, scale_layout, x, global_scales, codes, scales, &empty);
    if (st != MOE_OK || empty) return st;
    moe::LaunchCtx ctx;
    st = make_ctx(stream, &ctx);
    if (st != MOE_OK) return st;
    return from_cuda(moe::launch_quantize_nvfp4(ctx, x, groups, rows, hidden, global_scales, int(scale_layout), codes,
                                                scales));
}

moe_status_t moe_dequantize_nvfp4(const uint8_t* codes, const uint8_t* scales, int64_t groups, int64_t rows,
                                  int hidden, const float* global_scales, moe_scale_layout_t scale_layout,
                                  uint16_t* out, moe_stream_t stream) {
    bool empty;
    moe_status_t st = check_quant(groups, rows, hidden, scale_layout, out, global_scales, codes, scales, &empty);
    if (st != MOE_OK || empty) return st;
    moe::LaunchCtx ctx;
    st = make_ctx(stream, &ctx);
    if (st != MOE_OK) return st;
    return from_cuda(moe::launch_dequantize_nvfp4(ctx, codes, scales, groups, rows, hidden, global_scales,
                                                  int(scale_layout), out));
}

moe_status_t moe_expert_gemm(moe_mode_t mode, const uint8_t* a_codes, const uint8_t* a_scales,
                             moe_scale_layout_t scale_layout, int num_experts, int max_tokens_per_expert,
                             int64_t rows, int n, int k, const int64_t* seg_indptr, const int32_t* masked_m,
                             const uint8_t* w_codes, const uint8_t* w_scales, const float* alpha, uint16_t* out,
                             int32_t* dev_status, moe_stream_t stream) {
    moe_status_t st = check_gemm(mode, scale_layout, num_experts, max_tokens_per_expert, &rows, n, k, seg_indptr,
                                 masked_m, a_codes, a_scales, w_codes, w_scales, alpha, dev_status);
    if (st != MOE_OK) return st;
    if (rows == 0) return MOE_OK;
    if (!out || !aligned(out, 16)) return MOE_ERR_INVALID_ARG;
    moe::LaunchCtx ctx;
    st = make_ctx(stream, &ctx);
    if (st != MOE_OK) return st;
    const moe::ExpertGemm g{a_codes, a_scales, int(scale_layout), num_experts,
                            mode == MOE_MODE_MASKED ? max_tokens_per_expert : 0, rows, n, k, seg_indptr, masked_m,
                            w_codes, w_scales, alpha, out, 0.0f, nullptr, nullptr, dev_status};
    return from_cuda(moe::launch_expert_gemm(ctx, g));
}

moe_status_t moe_expert_gemm_swiglu(moe_mode_t mode, const uint8_t* a_codes, const uint8_t* a_scales,
                                    moe_scale_layout_t scale_layout, int num_experts, int max_tokens_per_expert,
                                    int64_t rows, int inter, int k, const int64_t* seg_indptr,
                                    const int32_t* masked_m, const uint8_t* w13_codes, const uint8_t* w13_scales,
                                    const float* alpha, float out_global_scale, uint8_t* out_codes,
                                    uint8_t* out_scales, int32_t* dev_status, moe_stream_t stream) {
    moe_status_t st = check_gemm(mode, scale_layout, num_experts, max_tokens_per_expert, &rows, inter, k, seg_indptr,
                                 masked_m, a_codes, a_scales, w13_codes, w13_scales, alpha, dev_status);
    if (st != MOE_OK) return st;
    if (inter % 64 != 0) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!out_codes || !out_scales || !aligned(out_codes, 16) || !aligned(out_scales, 4)) return MOE_ERR_INVALID_ARG;
    moe::LaunchCtx ctx;
    st = make_ctx(stream, &ctx);
    if (st != MOE_OK) return st;
    const moe::ExpertGemm g{a_codes, a_scales, int(scale_layout), num_experts,
                            mode == MOE_MODE_MASKED ? max_tokens_per_expert : 0, rows, inter, k, seg_indptr, masked_m,
                            w13_codes, w13_scales, alpha, nullptr, out_global_scale, out_codes, out_scales,
                            dev_status};
    return from_cuda(moe::launch_expert_gemm(ctx, g));
}

static moe_status_t check_layer_shape(int64_t T, int K, int H, int I, int E) {
    moe_status_t st = moe::check_shape(T, K, E);
    if (st != MOE_OK) return st;
    if (H <= 0 || I <= 0 || H % 16 != 0 || I % 16 != 0) return MOE_ERR_INVALID_ARG;
    if (T > MOE_LAYER_MAX_TOKENS || H > (1 << 20) || I > (1 << 20)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

size_t moe_layer_workspace_size(int64_t num_tokens, int topk, int hidden, int inter, int num_experts) {
    if (check_layer_shape(num_tokens, topk, hidden, inter, num_experts) != MOE_OK) return 0;
    return moe::few_tokens_workspace(num_tokens, topk, hidden, inter, num_experts);
}

moe_status_t moe_layer_few_tokens(const uint16_t* x, int64_t num_tokens, int hidden, int inter,
                                  const int32_t* topk_ids, const float* topk_weights, int topk, int num_experts,
                                  moe_quant_t weight_quant, const void* w13, const uint8_t* w13_scales,
                                  const float* alpha13, const void* w2, const uint8_t* w2_scales,
                                  const float* alpha2, uint16_t* out, void* workspace, size_t workspace_bytes,
                                  int32_t* dev_status, moe_stream_t stream) {
    moe_status_t st = check_layer_shape(num_tokens, topk, hidden, inter, num_experts);
    if (st != MOE_OK) return st;
    if (weight_quant != MOE_QUANT_NONE && weight_quant != MOE_QUANT_NVFP4_B16) return MOE_ERR_INVALID_ARG;
    const bool nvfp4 = weight_quant == MOE_QUANT_NVFP4_B16;
    if (nvfp4 && (hidden % 64 != 0 || inter % 64 != 0)) return MOE_ERR_INVALID_ARG;
    if (!dev_status || !aligned(dev_status, 4)) return MOE_ERR_INVALID_ARG;
    if (num_tokens == 0) return MOE_OK;
    if (!x || !topk_ids || !topk_weights || !w13 || !w2 || !out || !workspace) return MOE_ERR_INVALID_ARG;
    if (nvfp4 && (!w13_scales || !w2_scales)) return MOE_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(topk_ids, 4) || !aligned(topk_weights, 4) || !aligned(w13, 16) ||
        !aligned(w2, 16) || !aligned(w13_scales, 16) || !aligned(w2_scales, 16) || !aligned(alpha13, 4) ||
        !aligned(alpha2, 4) || !aligned(out, 16) || !aligned(workspace, 256))
        return MOE_ERR_INVALID_ARG;
    if (workspace_bytes < moe::few_tokens_workspace(num_tokens, topk, hidden, inter, num_experts))
        return MOE_ERR_INVALID_ARG;
    moe::LaunchCtx ctx;
    st = make_ctx(stream, &ctx);
    if (st != MOE_OK) return st;
    const moe::FewTokens a{x, int(num_tokens), hidden, inter, topk_ids, topk_weights, topk, num_experts, nvfp4, w13,
                           w13_scales, alpha13, w2, w2_scales, alpha2, out, workspace, dev_status};
    return from_cuda(moe::launch_few_tokens(ctx, a));
}

}  // extern "C"
