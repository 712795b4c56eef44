// block_launch.h -- host-side launch interface between block_abi.cu and the kernels of a MoE block's
// bf16 operators. Arguments arrive here already validated.
#pragma once

#include <cstddef>
#include <cstdint>

#include "moe_launch.h"

namespace moe {

// Which rows of a dispatched layout belong to which expert.
struct RowLayout {
    int E, M;              // M: masked capacity, 0 in normal mode
    int64_t rows;          // of the row buffers
    const int64_t* seg;    // normal mode
    const int32_t* count;  // masked_m
    int32_t* status;
};

// Products over the experts of a layout (expert_gemm_bf16.cu).
enum class RowOp { kPlain, kSwiglu, kDswiglu };
struct RowGemm {
    RowLayout rows;
    RowOp op;
    bool kn;                  // the weights are [E, k, n] (kDswiglu: always; kSwiglu: never)
    const uint16_t* a;        // [rows, k]
    int n, k;                 // columns of the result (kSwiglu, kDswiglu: inter), of a
    const uint16_t* w;        // kSwiglu: [E, 2, n, k]
    uint16_t* out;            // [rows, n]; kDswiglu: the gradient of gate_up [rows, 2n]
    uint16_t* gate_up;        // [rows, 2n]: kSwiglu: written, or null; kDswiglu: read
};
cudaError_t launch_row_gemm(const LaunchCtx& ctx, const RowGemm& g);

// Sums over an expert's rows (expert_wgrad_bf16.cu): over at most so many, so that every wait for one can be bounded.
constexpr int64_t kMostSummedRows = 1 << 26;
struct WeightGrad {
    RowLayout rows;
    const uint16_t* a;  // [rows, m]
    const uint16_t* b;  // [rows, n]
    int m, n;
    bool fp32, accumulate;
    void* out;  // [E, m, n]
};
cudaError_t launch_weight_grad(const LaunchCtx& ctx, const WeightGrad& g);

// combine_backward.cu
struct CombineGrad {
    bool masked;
    const uint16_t* grad;        // [T, H]
    const uint16_t* expert_out;  // null: no gradient of the weights
    int64_t T;
    int H, K, E, M;
    int64_t rows;                // of both row buffers (normal mode)
    const int32_t* ids;
    const int32_t* src2dst;
    const int64_t* seg;
    const float* w;
    uint16_t* grad_rows;         // or null
    float* grad_w;               // or null
    int32_t* status;
};
cudaError_t launch_combine_backward(const LaunchCtx& ctx, const CombineGrad& g);

// rmsnorm.cu
struct Norm {
    const uint16_t* x;
    const uint16_t* residual;  // or null
    const uint16_t* weight;
    float eps;
    int64_t T;
    int H;
    int quant;                 // MOE_QUANT_NONE, _FP8_G128 or _FP8_G128_UE8M0
    uint16_t* out;             // or null
    uint8_t* codes;
    void* scales;
    uint16_t* sum;             // or null
    float* rstd;               // or null
};
cudaError_t launch_rmsnorm(const LaunchCtx& ctx, const Norm& a);

struct NormGrad {
    const uint16_t* grad;
    const uint16_t* s;
    const uint16_t* weight;
    const float* rstd;
    const uint16_t* grad_sum;  // or null
    int64_t T;
    int H;
    uint16_t* grad_x;
    float* grad_weight;
    float* partial;            // [norm_backward_blocks(T, H), H]
};
int norm_backward_blocks(int64_t T, int H);
cudaError_t launch_rmsnorm_backward(const LaunchCtx& ctx, const NormGrad& a);

}  // namespace moe
