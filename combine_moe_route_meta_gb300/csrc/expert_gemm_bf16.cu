// expert_gemm_bf16.cu -- the products of a dispatched layout's bf16 rows with their expert's weights.
//
//   plain     out[r, j] = sum_k a[r, k] w(e, j, k), weights [E, n, k] or [E, k, n]
//   SwiGLU    h = up * silu(gate) of two such products
//   dSwiGLU   the gradient of gate and up from such a product
//
// One block takes 64 rows x 64 columns of one expert; a thread 4 x 4 of them, in fp32.
#include <cstdint>

#include "block_launch.h"
#include "expert_rows.cuh"

namespace moe {
namespace {

constexpr int kTile = 64, kStep = 16, kThreads = 256;

struct RowTile {
    int e, rows;
    int64_t row0;
};

// The block's row tile: number t of all experts', found by one thread. e = -1: there is none.
__device__ RowTile find_row_tile(const RowLayout& l, int t) {
    int64_t wide = 0;
    for (int e = 0; e < l.E; e++) wide += (expert_rows(l, e).count + 255) / 256;
    if (wide > l.rows / 256 + l.E) {
        set_status(l.status, MOE_ERR_INVALID_ARG);
        return RowTile{-1, 0, 0};
    }
    for (int e = 0; e < l.E; e++) {
        const RowSpan r = expert_rows(l, e);
        const int tiles = int((int64_t(r.count) + kTile - 1) / kTile);
        if (t < tiles) return RowTile{e, min(kTile, r.count - t * kTile), r.base + int64_t(t) * kTile};
        t -= tiles;
    }
    return RowTile{-1, 0, 0};
}

template <RowOp OP, bool KN>
__global__ void __launch_bounds__(kThreads) row_gemm_kernel(RowGemm g) {
    constexpr int kHalves = OP == RowOp::kSwiglu ? 2 : 1;
    __shared__ float sa[kStep][kTile + 1], sw[kHalves][kStep][kTile + 1];
    __shared__ RowTile tile;
    pdl_wait();
    if (threadIdx.x == 0) tile = find_row_tile(g.rows, blockIdx.y);
    __syncthreads();
    if (tile.e < 0) return;
    const int n0 = blockIdx.x * kTile, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    const uint16_t* w = g.w + int64_t(tile.e) * kHalves * g.n * g.k;
    float acc[kHalves][4][4] = {};
    for (int k0 = 0; k0 < g.k; k0 += kStep) {
        for (int i = threadIdx.x; i < kTile * kStep; i += kThreads) {
            const int r = i / kStep, k = k0 + i % kStep;
            sa[i % kStep][r] = r < tile.rows && k < g.k ? bf16_lo(g.a[(tile.row0 + r) * g.k + k]) : 0.0f;
            for (int h = 0; h < kHalves; h++) {
                const int kk = KN ? i / kTile : i % kStep, j = KN ? i % kTile : i / kStep;
                const bool in = k0 + kk < g.k && n0 + j < g.n;
                const int64_t at = KN ? int64_t(k0 + kk) * g.n + n0 + j : (int64_t(h) * g.n + n0 + j) * g.k + k0 + kk;
                sw[h][kk][j] = in ? bf16_lo(w[at]) : 0.0f;
            }
        }
        __syncthreads();
        for (int k = 0; k < kStep; k++)
            for (int h = 0; h < kHalves; h++)
                for (int i = 0; i < 4; i++)
                    for (int j = 0; j < 4; j++)
                        acc[h][i][j] = fmaf(sa[k][ty * 4 + i], sw[h][k][tx * 4 + j], acc[h][i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; i++) {
        const int64_t r = tile.row0 + ty * 4 + i;
        if (ty * 4 + i >= tile.rows) break;
        for (int j = 0; j < 4; j++) {
            const int c = n0 + tx * 4 + j;
            if (c >= g.n) break;
            const float v = acc[0][i][j];
            if constexpr (OP == RowOp::kPlain) {
                g.out[r * g.n + c] = uint16_t(pack_bf16x2(v, 0.0f));
            } else if constexpr (OP == RowOp::kSwiglu) {
                const float up = acc[kHalves - 1][i][j];
                g.out[r * g.n + c] = uint16_t(pack_bf16x2(swiglu(v, up), 0.0f));
                if (g.gate_up) {
                    g.gate_up[r * 2 * g.n + c] = uint16_t(pack_bf16x2(v, 0.0f));
                    g.gate_up[(r * 2 + 1) * g.n + c] = uint16_t(pack_bf16x2(up, 0.0f));
                }
            } else {
                const int64_t at = r * 2 * g.n + c;
                float dgate, dup;
                dswiglu(bf16_lo(g.gate_up[at]), bf16_lo(g.gate_up[at + g.n]), v, &dgate, &dup);
                g.out[at] = uint16_t(pack_bf16x2(dgate, 0.0f));
                g.out[at + g.n] = uint16_t(pack_bf16x2(dup, 0.0f));
            }
        }
    }
}

template <RowOp OP, bool KN>
cudaError_t launch(const LaunchCtx& ctx, const RowGemm& g) {
    const int64_t tiles = g.rows.rows / kTile + g.rows.E;
    if (tiles > 65535) return cudaErrorInvalidValue;
    return launch_pdl(ctx, row_gemm_kernel<OP, KN>, dim3(unsigned((g.n + kTile - 1) / kTile), unsigned(tiles)),
                      dim3(kThreads), 0, g);
}

}  // namespace

cudaError_t launch_row_gemm(const LaunchCtx& ctx, const RowGemm& g) {
    if (g.op == RowOp::kSwiglu) return launch<RowOp::kSwiglu, false>(ctx, g);
    if (g.op == RowOp::kDswiglu) return launch<RowOp::kDswiglu, true>(ctx, g);
    return g.kn ? launch<RowOp::kPlain, true>(ctx, g) : launch<RowOp::kPlain, false>(ctx, g);
}

}  // namespace moe
