// experts_launch.h -- host-side launch interface between experts_abi.cu and the kernels of the
// expert operators. Arguments arrive here already validated.
#pragma once

#include <cstddef>
#include <cstdint>

#include "moe_launch.h"

namespace moe {

cudaError_t launch_quantize_nvfp4(const LaunchCtx& ctx, const uint16_t* x, int64_t G, int64_t R, int H,
                                  const float* gs, int scale_layout, uint8_t* codes, uint8_t* scales);
cudaError_t launch_dequantize_nvfp4(const LaunchCtx& ctx, const uint8_t* codes, const uint8_t* scales, int64_t G,
                                    int64_t R, int H, const float* gs, int scale_layout, uint16_t* out);

// The rows of a dispatched layout and the product over its experts (expert_gemm.cu).
struct ExpertGemm {
    const uint8_t* a;        // [rows, k/2]
    const uint8_t* a_sf;     // [rows, k/16] in scale_layout
    int scale_layout;        // of a_sf and, with SwiGLU, of h_sf
    int E, M;                // M: masked capacity, 0 in normal mode
    int64_t rows;            // rows of a and of the output
    int n, k;                // columns of w (SwiGLU: inter gate and inter up columns, n = inter)
    const int64_t* seg;      // normal mode
    const int32_t* count;    // masked_m
    const uint8_t* w;        // [E, n, k/2]; SwiGLU [E, 2, n, k/2]
    const uint8_t* w_sf;     // per expert (and half) tiles of [roundup(n, 128), k/16]
    const float* alpha;      // [E] or null
    uint16_t* out;           // [rows, n] bf16, null with SwiGLU
    float h_scale;           // SwiGLU: global scale of h
    uint8_t* h;              // SwiGLU: [rows, n/2]
    uint8_t* h_sf;           // SwiGLU: [rows, n/16]
    int32_t* status;
};
cudaError_t launch_expert_gemm(const LaunchCtx& ctx, const ExpertGemm& g);

struct FewTokens {
    const uint16_t* x;
    int T, H, I;
    const int32_t* ids;
    const float* w;
    int K, E;
    bool nvfp4;
    const void* w13;
    const uint8_t* w13_sf;
    const float* alpha13;
    const void* w2;
    const uint8_t* w2_sf;
    const float* alpha2;
    uint16_t* out;
    void* workspace;
    int32_t* status;
};
size_t few_tokens_workspace(int64_t T, int K, int H, int I, int E);
cudaError_t launch_few_tokens(const LaunchCtx& ctx, const FewTokens& a);

}  // namespace moe
