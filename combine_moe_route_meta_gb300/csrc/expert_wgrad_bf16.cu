// expert_wgrad_bf16.cu -- the gradient of the experts' weights: out[e, i, j] (+)= sum_r a[r, i] b[r, j] over the rows
// of each expert.
//
// One block takes 64 x 64 of one expert's results; a thread 4 x 4 of them, in fp32.
#include <cstdint>

#include "block_launch.h"
#include "expert_rows.cuh"

namespace moe {
namespace {

constexpr int kTile = 64, kStep = 16, kThreads = 256;

__global__ void __launch_bounds__(kThreads) weight_grad_kernel(WeightGrad g, int tiles_n) {
    __shared__ float sa[kStep][kTile + 1], sb[kStep][kTile + 1];
    pdl_wait();
    const int e = blockIdx.y, m0 = int(blockIdx.x) / tiles_n * kTile, n0 = int(blockIdx.x) % tiles_n * kTile;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    const RowSpan span = expert_rows(g.rows, e);
    float acc[4][4] = {};
    for (int r0 = 0; r0 < span.count; r0 += kStep) {
        for (int i = threadIdx.x; i < kTile * kStep; i += kThreads) {
            const int r = i / kTile, c = i % kTile;
            const bool in = r0 + r < span.count;
            sa[r][c] = in && m0 + c < g.m ? bf16_lo(g.a[(span.base + r0 + r) * g.m + m0 + c]) : 0.0f;
            sb[r][c] = in && n0 + c < g.n ? bf16_lo(g.b[(span.base + r0 + r) * g.n + n0 + c]) : 0.0f;
        }
        __syncthreads();
        for (int r = 0; r < kStep; r++)
            for (int i = 0; i < 4; i++)
                for (int j = 0; j < 4; j++) acc[i][j] = fmaf(sa[r][ty * 4 + i], sb[r][tx * 4 + j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; i++)
        for (int j = 0; j < 4; j++) {
            const int r = m0 + ty * 4 + i, c = n0 + tx * 4 + j;
            if (r >= g.m || c >= g.n) continue;
            const int64_t at = (int64_t(e) * g.m + r) * g.n + c;
            if (g.fp32) {
                float* out = static_cast<float*>(g.out) + at;
                *out = g.accumulate ? *out + acc[i][j] : acc[i][j];
            } else {
                uint16_t* out = static_cast<uint16_t*>(g.out) + at;
                *out = uint16_t(pack_bf16x2(g.accumulate ? bf16_lo(*out) + acc[i][j] : acc[i][j], 0.0f));
            }
        }
}

}  // namespace

cudaError_t launch_weight_grad(const LaunchCtx& ctx, const WeightGrad& g) {
    const int tiles_m = (g.m + kTile - 1) / kTile, tiles_n = (g.n + kTile - 1) / kTile;
    return launch_pdl(ctx, weight_grad_kernel, dim3(unsigned(tiles_m * tiles_n), unsigned(g.rows.E)), dim3(kThreads), 0,
                      g, tiles_n);
}

}  // namespace moe
