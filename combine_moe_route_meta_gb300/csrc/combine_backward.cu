// combine_backward.cu -- the gradient of the combine:
//   grad_rows[row(t, k), :] = bf16(w[t, k] * grad[t, :]),  grad_w[t, k] = sum_h grad[t, h] * expert_out[row(t, k), h]
//
// One block of four warps a token. A warp takes slices of 512 columns: a lane two runs of 8 columns, 256 columns apart, so
// that a warp's 16-byte accesses cover 512 contiguous bytes. The slice of grad is read once for all k; up to 8 rows of
// expert_out are in flight before the first is used. The dot products are summed in fp32: a lane's 16 columns of each
// slice, the lanes by halves, the warps in order, so a result depends on the arguments alone.
// Bound by DRAM: 16384 tokens top-8, 4096 columns: 322 us, 6.75 TB/s, the copy bandwidth.
#include <cstdint>

#include "block_launch.h"
#include "moe_device.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;
constexpr int kSlice = 512;
constexpr int kBatch = 8;  // rows in flight

// grad_rows may be expert_out: a plain load, not one through the read-only path
__device__ __forceinline__ uint4 ld_v4(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ uint4 scaled(const float* g, float w) {
    return make_uint4(pack_bf16x2(w * g[0], w * g[1]), pack_bf16x2(w * g[2], w * g[3]), pack_bf16x2(w * g[4], w * g[5]),
                      pack_bf16x2(w * g[6], w * g[7]));
}

// The row of slot `lane` of token t, -1: none.
__device__ __forceinline__ int64_t slot_row(const CombineGrad& a, int64_t t, int lane) {
    if (lane >= a.K) return -1;
    const int d = __ldg(a.src2dst + t * a.K + lane);
    if (d < 0) return -1;
    if (a.masked) {
        const int e = __ldg(a.ids + t * a.K + lane);
        if (e < 0 || e >= a.E) {
            set_status(a.status, MOE_ERR_BAD_EXPERT_ID);
            return -1;
        }
        const int64_t rank = d - __ldg(a.seg + e);
        return rank >= 0 && rank < a.M ? int64_t(e) * a.M + rank : -1;
    }
    if (d < a.rows) return d;
    set_status(a.status, MOE_ERR_INVALID_ARG);
    return -1;
}

__global__ void __launch_bounds__(kWarps * 32) combine_backward_kernel(CombineGrad a) {
    __shared__ float sums[kWarps][MOE_MAX_TOPK];
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, H = a.H;
    const int64_t t = blockIdx.x;
    const int64_t my_row = slot_row(a, t, lane);
    const float my_w = lane < a.K && a.w ? __ldg(a.w + t * a.K + lane) : 0.0f;
    for (int k0 = 0; k0 < a.K; k0 += kBatch) {
        int64_t row[kBatch];
        float w[kBatch], acc[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; j++) {
            row[j] = __shfl_sync(kFullMask, my_row, (k0 + j) & 31);
            w[j] = __shfl_sync(kFullMask, my_w, (k0 + j) & 31);
            acc[j] = 0.0f;
        }
        for (int c = warp * kSlice; c < H; c += kWarps * kSlice) {
            const int c0 = c + lane * 8, c1 = c0 + kSlice / 2;
            if (c0 >= H) continue;
            const bool two = c1 < H;
            const uint4 zero = make_uint4(0, 0, 0, 0);
            uint4 v[kBatch][2];
            if (a.expert_out) {
#pragma unroll
                for (int j = 0; j < kBatch; j++) {
                    const uint16_t* p = a.expert_out + row[j] * H;
                    v[j][0] = row[j] >= 0 ? ld_v4(p + c0) : zero;
                    v[j][1] = row[j] >= 0 && two ? ld_v4(p + c1) : zero;
                }
            }
            float g[16];
            unpack8(ld_stream_v4(a.grad + t * H + c0), g);
            unpack8(two ? ld_stream_v4(a.grad + t * H + c1) : zero, g + 8);
#pragma unroll
            for (int j = 0; j < kBatch; j++) {
                if (row[j] < 0) continue;
                if (a.expert_out) {
                    float f[16];
                    unpack8(v[j][0], f);
                    unpack8(v[j][1], f + 8);
#pragma unroll
                    for (int i = 0; i < 16; i++) acc[j] = fmaf(g[i], f[i], acc[j]);
                }
                if (a.grad_rows) {
                    uint16_t* p = a.grad_rows + row[j] * H;
                    st_v4(p + c0, scaled(g, w[j]));
                    if (two) st_v4(p + c1, scaled(g + 8, w[j]));
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kBatch; j++) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) acc[j] += __shfl_xor_sync(kFullMask, acc[j], o);
            if (lane == 0 && k0 + j < a.K) sums[warp][k0 + j] = acc[j];
        }
    }
    if (!a.grad_w) return;
    __syncthreads();
    if (threadIdx.x < unsigned(a.K)) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kWarps; i++) s += sums[i][threadIdx.x];
        a.grad_w[t * a.K + threadIdx.x] = s;
    }
}

}  // namespace

cudaError_t launch_combine_backward(const LaunchCtx& ctx, const CombineGrad& a) {
    return launch_pdl(ctx, combine_backward_kernel, dim3(unsigned(a.T)), dim3(kWarps * 32), 0, a);
}

}  // namespace moe
