// moe_layer.cu -- a whole MoE layer for a few tokens in two kernels.
//
//   gate_up:  h(t, k) = silu(gate) * up of expert topk_ids[t, k] on token t   -> workspace, fp32 [T*K, I]
//   down:     out[t] = bf16(sum_k topk_weights[t, k] * alpha2[e] * W2[e] h(t, k))
//
// One warp per output value (pair and row of w13, token and row of w2).
#include <algorithm>
#include <cstdint>

#include "expert_rows.cuh"
#include "experts_launch.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

// dot of row `row` of matrix m (rows x k) with v, over one lane's blocks of 16
template <bool NVFP4, typename V>
__device__ __forceinline__ float row_dot(const void* w, const uint8_t* sf, int64_t m, int rows, int row, int k,
                                         const V* v, int lane) {
    float s = 0.0f;
    const int C = k / 16, rp = (rows + 127) / 128 * 128;
    for (int c = lane; c < C; c += 32) {
        float f[16];
        if (NVFP4) {
            const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(w) + ((m * rows + row) * C + c) * 8);
            const float sc = e4m3_value(sf[m * rp * C + swizzled_128x4_index(row, c, C)]);
            for (int j = 0; j < 16; j++) f[j] = sc * e2m1_value(((j < 8 ? q.x : q.y) >> (4 * (j & 7))) & 15u);
        } else {
            const uint16_t* p = static_cast<const uint16_t*>(w) + (m * rows + row) * int64_t(k) + c * 16;
            unpack8(ld_stream_v4(p), f);
            unpack8(ld_stream_v4(p + 8), f + 8);
        }
        for (int j = 0; j < 16; j++) {
            if constexpr (sizeof(V) == 2)
                s = fmaf(f[j], bf16_lo(v[c * 16 + j]), s);
            else
                s = fmaf(f[j], v[c * 16 + j], s);
        }
    }
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(kFullMask, s, o);
    return s;
}

template <bool NVFP4>
__global__ void __launch_bounds__(kThreads) few_tokens_gate_up_plain_kernel(FewTokens a) {
    pdl_wait();
    const int lane = threadIdx.x & 31, pair = blockIdx.y;
    const int i = int(blockIdx.x) * (kThreads / 32) + int(threadIdx.x >> 5);
    const int e = __ldg(a.ids + pair);
    if (e < 0 || e >= a.E) {
        if (e != -1 && i == 0 && lane == 0) set_status(a.status, MOE_ERR_BAD_EXPERT_ID);
        return;
    }
    if (i >= a.I) return;
    const uint16_t* x = a.x + int64_t(pair / a.K) * a.H;
    const float alpha = a.alpha13 ? __ldg(a.alpha13 + e) : 1.0f;
    const int64_t m = NVFP4 ? int64_t(e) * 2 : e;
    float g, u;
    if (NVFP4) {
        g = row_dot<true>(a.w13, a.w13_sf, m, a.I, i, a.H, x, lane);
        u = row_dot<true>(a.w13, a.w13_sf, m + 1, a.I, i, a.H, x, lane);
    } else {
        g = row_dot<false>(a.w13, nullptr, m, 2 * a.I, i, a.H, x, lane);
        u = row_dot<false>(a.w13, nullptr, m, 2 * a.I, a.I + i, a.H, x, lane);
    }
    if (lane == 0) static_cast<float*>(a.workspace)[int64_t(pair) * a.I + i] = swiglu(alpha * g, alpha * u);
}

template <bool NVFP4>
__global__ void __launch_bounds__(kThreads) few_tokens_down_plain_kernel(FewTokens a) {
    pdl_wait();
    const int lane = threadIdx.x & 31, t = blockIdx.y;
    const int r = int(blockIdx.x) * (kThreads / 32) + int(threadIdx.x >> 5);
    if (r >= a.H) return;
    float y = 0.0f;
    for (int k = 0; k < a.K; k++) {
        const int pair = t * a.K + k, e = __ldg(a.ids + pair);
        if (e < 0 || e >= a.E) continue;
        const float* h = static_cast<const float*>(a.workspace) + int64_t(pair) * a.I;
        const float d = row_dot<NVFP4>(a.w2, a.w2_sf, e, a.H, r, a.I, h, lane);
        y = fmaf(__ldg(a.w + pair) * (a.alpha2 ? __ldg(a.alpha2 + e) : 1.0f), d, y);
    }
    if (lane == 0) a.out[int64_t(t) * a.H + r] = uint16_t(pack_bf16x2(y, 0.0f));
}

}  // namespace

size_t few_tokens_workspace(int64_t T, int K, int, int I, int) { return size_t(T) * K * I * sizeof(float); }

cudaError_t launch_few_tokens(const LaunchCtx& ctx, const FewTokens& a) {
    const dim3 g1(unsigned((a.I + 7) / 8), unsigned(a.T * a.K)), g2(unsigned((a.H + 7) / 8), unsigned(a.T));
    cudaError_t err = launch_pdl(
        ctx, a.nvfp4 ? few_tokens_gate_up_plain_kernel<true> : few_tokens_gate_up_plain_kernel<false>, g1,
        dim3(kThreads), 0, a);
    if (err != cudaSuccess) return err;
    return launch_pdl(ctx, a.nvfp4 ? few_tokens_down_plain_kernel<true> : few_tokens_down_plain_kernel<false>, g2,
                      dim3(kThreads), 0, a);
}

}  // namespace moe
