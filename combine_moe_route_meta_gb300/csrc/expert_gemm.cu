// expert_gemm.cu -- the product of a dispatched layout's NVFP4 rows with their expert's weights.
//
//   out[r, n] = bf16(alpha[e] * sum_k a[r, k] w[e, n, k])
//   SwiGLU:  h = silu(gate) * up of two such products, quantised to NVFP4
//
// Plain tiles: a block computes 64 columns of one expert (SwiGLU: 32 gate and the 32 up columns beside
// them) for its rows, 64 at a time, from 64-deep slices decoded to fp32 in shared memory.
#include <cstdint>

#include "expert_rows.cuh"
#include "experts_launch.h"

namespace moe {
namespace {

constexpr int kTile = 64;
constexpr int kThreads = 256;

// 16 values of block `c` of a row into dst[0..15] (stride kTile + 1)
__device__ __forceinline__ void decode16(const uint8_t* codes, uint32_t sf, float* dst) {
    const uint2 q = *reinterpret_cast<const uint2*>(codes);
    const float s = e4m3_value(sf);
#pragma unroll
    for (int j = 0; j < 16; j++) {
        const uint32_t w = j < 8 ? q.x : q.y;
        dst[j * (kTile + 1)] = e2m1_value((w >> (4 * (j & 7))) & 15u) * s;
    }
}

template <bool SWIGLU>
__global__ void __launch_bounds__(kThreads) expert_gemm_plain_kernel(ExpertGemm a) {
    __shared__ float sa[kTile][kTile + 1];  // [k][row]
    __shared__ float sb[kTile][kTile + 1];  // [k][column]
    pdl_wait();
    const int e = blockIdx.y;
    const RowSpan span = expert_rows(a, e);
    const int C = a.k / 16, np = (a.n + 127) / 128 * 128;
    const int n0 = blockIdx.x * (SWIGLU ? kTile / 2 : kTile);
    const int tid = threadIdx.x, tr = tid / 16, tc = tid % 16;
    const float alpha = a.alpha ? __ldg(a.alpha + e) : 1.0f;

    for (int m0 = 0; m0 < span.count; m0 += kTile) {
        float acc[4][4] = {};
        for (int k0 = 0; k0 < a.k; k0 += kTile) {
            const int row = tid / 4, blk = tid % 4, c = k0 / 16 + blk;
            __syncthreads();
            if (m0 + row < span.count) {
                const int64_t r = span.base + m0 + row;
                decode16(a.a + (r * C + c) * 8, a.a_sf[act_sf_index(a.scale_layout, r, c, C)], &sa[blk * 16][row]);
            } else {
                for (int j = 0; j < 16; j++) sa[blk * 16 + j][row] = 0.0f;
            }
            const int half = SWIGLU ? row / (kTile / 2) : 0;
            const int n = n0 + (SWIGLU ? row % (kTile / 2) : row);
            if (n < a.n) {
                const int64_t m = SWIGLU ? int64_t(e) * 2 + half : e;  // weight matrix
                decode16(a.w + ((m * a.n + n) * C + c) * 8, a.w_sf[m * np * C + swizzled_128x4_index(n, c, C)],
                         &sb[blk * 16][row]);
            } else {
                for (int j = 0; j < 16; j++) sb[blk * 16 + j][row] = 0.0f;
            }
            __syncthreads();
            for (int k = 0; k < kTile; k++)
#pragma unroll
                for (int i = 0; i < 4; i++)
#pragma unroll
                    for (int j = 0; j < 4; j++) acc[i][j] = fmaf(sa[k][tr * 4 + i], sb[k][tc * 4 + j], acc[i][j]);
        }
        if (!SWIGLU) {
            for (int i = 0; i < 4; i++)
                for (int j = 0; j < 4; j++)
                    if (m0 + tr * 4 + i < span.count && n0 + tc * 4 + j < a.n)
                        a.out[(span.base + m0 + tr * 4 + i) * a.n + n0 + tc * 4 + j] =
                            uint16_t(pack_bf16x2(alpha * acc[i][j], 0.0f));
        } else {
            __syncthreads();
            for (int i = 0; i < 4; i++)
                for (int j = 0; j < 4; j++) sa[tr * 4 + i][tc * 4 + j] = alpha * acc[i][j];
            __syncthreads();
            const int row = tid / 2, blk = tid % 2;  // 64 rows x 2 blocks of 16
            if (tid < 128 && m0 + row < span.count && n0 + blk * 16 < a.n) {
                uint32_t w[8];
                for (int p = 0; p < 8; p++)
                    w[p] = 0;
                float h[16], amax = 0.0f;
                for (int j = 0; j < 16; j++) {
                    h[j] = swiglu(sa[row][blk * 16 + j], sa[row][kTile / 2 + blk * 16 + j]);
                    amax = fmaxf(amax, fabsf(h[j]));
                }
                const uint32_t sf = e4m3x2(__fmul_rn(__fdiv_rn(amax, 6.0f), a.h_scale), 0.0f) & 0xffu;
                const float sff = e4m3_value(sf);
                if (sff != 0.0f) {
                    const float rs = __fdiv_rn(a.h_scale, sff);
                    for (int p = 0; p < 8; p++) w[p] = e2m1x2(__fmul_rn(h[2 * p], rs), __fmul_rn(h[2 * p + 1], rs));
                }
                const int64_t r = span.base + m0 + row;
                const int c = n0 / 16 + blk, hc = a.n / 16;
                st_v2(a.h + (r * hc + c) * 8, make_uint2(w[0] | w[1] << 8 | w[2] << 16 | w[3] << 24,
                                                         w[4] | w[5] << 8 | w[6] << 16 | w[7] << 24));
                a.h_sf[act_sf_index(a.scale_layout, r, c, hc)] = uint8_t(sf);
            }
            __syncthreads();
        }
    }
}

}  // namespace

cudaError_t launch_expert_gemm(const LaunchCtx& ctx, const ExpertGemm& g) {
    const bool swiglu = g.out == nullptr;
    const int cols = swiglu ? kTile / 2 : kTile;
    const dim3 grid(unsigned((g.n + cols - 1) / cols), unsigned(g.E));
    return launch_pdl(ctx, swiglu ? expert_gemm_plain_kernel<true> : expert_gemm_plain_kernel<false>, grid,
                      dim3(kThreads), 0, g);
}

}  // namespace moe
