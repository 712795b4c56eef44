// rmsnorm.cu -- root-mean-square norm of x + residual, in bf16 and in FP8 with a scale for each 128 values, and its
// gradient.
//
// A row stays in registers between its one reading and its one writing. A lane has runs of 8 columns, threads next to
// each other neighbouring runs, so accesses are of 16 bytes and the 128 values of an FP8 group lie in 16 neighbouring
// lanes. Rows of up to 1024 columns are a warp's, longer ones a block's. The gradient of the weight is a sum over rows:
// each of at most kGradBlocks blocks sums its rows in registers and writes one line of partial sums; a second kernel adds
// the lines in order.
#include <cstdint>

#include "block_launch.h"
#include "dispatch_slice.cuh"
#include "moe_device.cuh"

namespace moe {
namespace {

constexpr int kGradBlocks = 304;
constexpr int kWarpRows = 4;  // rows of a block whose warps have a row each

__device__ __forceinline__ uint4 ld_v4(const void* p) {  // of what may be written in place
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint4 pack8(const float* f) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// The sum of v over the row's threads: a warp, or the block. `turn` alternates from call to call.
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float (*part)[32], int turn) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    if constexpr (WARP) return v;
    const int warps = blockDim.x / 32;
    if (threadIdx.x % 32 == 0) part[turn][threadIdx.x / 32] = v;
    __syncthreads();
    v = int(threadIdx.x % 32) < warps ? part[turn][threadIdx.x % 32] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}

template <int V, int QUANT, bool WARP>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(Norm a) {
    __shared__ float part[1][32];
    pdl_wait();
    const int64_t t = WARP ? int64_t(blockIdx.x) * kWarpRows + threadIdx.x / 32 : blockIdx.x;
    const int lane = WARP ? threadIdx.x % 32 : threadIdx.x, lanes = WARP ? 32 : blockDim.x;
    if (WARP && t >= a.T) return;
    const int64_t row = t * a.H;
    float s[V][8], square = 0.0f;
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int c = (v * lanes + lane) * 8;
        const bool in = c < a.H;
        unpack8(in ? ld_v4(a.x + row + c) : make_uint4(0, 0, 0, 0), s[v]);
        if (a.residual && in) {
            float r[8];
            unpack8(ld_v4(a.residual + row + c), r);
#pragma unroll
            for (int j = 0; j < 8; j++) s[v][j] += r[j];
            // the norm is of the sum as it is stored, rounded: what the next layer and the gradient see
            const uint4 sum = pack8(s[v]);
            unpack8(sum, s[v]);
            if (a.sum) st_v4(a.sum + row + c, sum);
        }
#pragma unroll
        for (int j = 0; j < 8; j++) square = fmaf(s[v][j], s[v][j], square);
    }
    square = row_sum<WARP>(square, part, 0);
    const float r = __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(square, float(a.H)), a.eps)));
    if (a.rstd && lane == 0) a.rstd[t] = r;
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int c = (v * lanes + lane) * 8;
        const bool in = c < a.H;
        float y[8];
        unpack8(in ? __ldg(reinterpret_cast<const uint4*>(a.weight + c)) : make_uint4(0, 0, 0, 0), y);
#pragma unroll
        for (int j = 0; j < 8; j++) y[j] = __fmul_rn(__fmul_rn(s[v][j], r), y[j]);
        if (a.out && in) st_v4(a.out + row + c, pack8(y));
        if constexpr (QUANT != MOE_QUANT_NONE) {
            // the unrounded values: one rounding to 8 bits, not two
            float amax = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; j++) amax = fmaxf(amax, fabsf(y[j]));
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, o));
            const float sc = __fdiv_rn(fmaxf(amax, 1e-10f), 448.0f);
            uint32_t q[2];
            if constexpr (QUANT == MOE_QUANT_FP8_G128) {
                const float inv = __frcp_rn(sc);
#pragma unroll
                for (int j = 0; j < 8; j++) y[j] = div_by_scale(y[j], sc, inv);
                if (in && lane % 16 == 0) static_cast<float*>(a.scales)[t * (a.H / 128) + c / 128] = sc;
            } else {
                const uint32_t bits = __float_as_uint(sc);
                const uint32_t ex = (bits >> 23) + ((bits & 0x7fffffu) ? 1u : 0u);
                const float inv = __uint_as_float((254u - ex) << 23);  // of a power of two: exact
#pragma unroll
                for (int j = 0; j < 8; j++) y[j] = __fmul_rn(y[j], inv);
                if (in && lane % 16 == 0) static_cast<uint8_t*>(a.scales)[t * (a.H / 128) + c / 128] = uint8_t(ex);
            }
#pragma unroll
            for (int j = 0; j < 2; j++) q[j] = e4m3x2(y[4 * j], y[4 * j + 1]) | e4m3x2(y[4 * j + 2], y[4 * j + 3]) << 16;
            if (in) st_v2(a.codes + row + c, make_uint2(q[0], q[1]));
        }
    }
}

template <int V, bool WARP>
__global__ void __launch_bounds__(1024) rmsnorm_backward_kernel(NormGrad a) {
    __shared__ float part[2][32];
    extern __shared__ float lines[];  // WARP: [kWarpRows][H]
    pdl_wait();
    const int lane = WARP ? threadIdx.x % 32 : threadIdx.x, lanes = WARP ? 32 : blockDim.x;
    const int64_t first = WARP ? int64_t(blockIdx.x) * kWarpRows + threadIdx.x / 32 : blockIdx.x;
    const int64_t step = WARP ? int64_t(gridDim.x) * kWarpRows : gridDim.x;
    float acc[V][8] = {};
    int turn = 0;
    for (int64_t t = first; t < a.T; t += step, turn ^= 1) {
        const int64_t row = t * a.H;
        const float r = __ldg(a.rstd + t);
        float hat[V][8], gw[V][8], dot = 0.0f;
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int c = (v * lanes + lane) * 8;
            const bool in = c < a.H;
            const uint4 zero = make_uint4(0, 0, 0, 0);
            float w[8];
            unpack8(in ? ld_v4(a.s + row + c) : zero, hat[v]);
            unpack8(in ? ld_v4(a.grad + row + c) : zero, gw[v]);
            unpack8(in ? __ldg(reinterpret_cast<const uint4*>(a.weight + c)) : zero, w);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                hat[v][j] *= r;
                acc[v][j] = fmaf(gw[v][j], hat[v][j], acc[v][j]);
                gw[v][j] *= w[j];
                dot = fmaf(gw[v][j], hat[v][j], dot);
            }
        }
        const float mean = __fdiv_rn(row_sum<WARP>(dot, part, turn), float(a.H));
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int c = (v * lanes + lane) * 8;
            if (c >= a.H) continue;
            float d[8], more[8];
            unpack8(a.grad_sum ? ld_v4(a.grad_sum + row + c) : make_uint4(0, 0, 0, 0), more);
#pragma unroll
            for (int j = 0; j < 8; j++) d[j] = fmaf(r, fmaf(-mean, hat[v][j], gw[v][j]), more[j]);
            st_v4(a.grad_x + row + c, pack8(d));
        }
    }
    float* line = a.partial + int64_t(blockIdx.x) * a.H;
    if constexpr (WARP) {
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int c = (v * 32 + lane) * 8;
            if (c >= a.H) continue;
            for (int j = 0; j < 8; j++) lines[threadIdx.x / 32 * a.H + c + j] = acc[v][j];
        }
        __syncthreads();
        for (int c = threadIdx.x; c < a.H; c += blockDim.x) {
            float sum = 0.0f;
            for (int i = 0; i < kWarpRows; i++) sum += lines[i * a.H + c];
            line[c] = sum;
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int c = (v * lanes + lane) * 8;
            if (c >= a.H) continue;
            *reinterpret_cast<float4*>(line + c) = make_float4(acc[v][0], acc[v][1], acc[v][2], acc[v][3]);
            *reinterpret_cast<float4*>(line + c + 4) = make_float4(acc[v][4], acc[v][5], acc[v][6], acc[v][7]);
        }
    }
}

// grad_weight[c] = the sum of `n` lines: 8 threads a column, then these in order.
__global__ void __launch_bounds__(256) add_lines_kernel(const float* lines, int n, int H, float* out) {
    __shared__ float sums[8][32];
    pdl_wait();
    const int c = blockIdx.x * 32 + threadIdx.x % 32, part = threadIdx.x / 32;
    float s = 0.0f;
    if (c < H)
#pragma unroll 8
        for (int i = part; i < n; i += 8) s += lines[int64_t(i) * H + c];
    sums[part][threadIdx.x % 32] = s;
    __syncthreads();
    if (part != 0 || c >= H) return;
#pragma unroll
    for (int i = 1; i < 8; i++) s += sums[i][threadIdx.x];
    out[c] = s;
}

template <int V, bool WARP>
cudaError_t launch_norm(const LaunchCtx& ctx, const Norm& a, int threads) {
    const unsigned grid = unsigned(WARP ? (a.T + kWarpRows - 1) / kWarpRows : a.T);
    if (a.quant == MOE_QUANT_NONE)
        return launch_pdl(ctx, rmsnorm_kernel<V, MOE_QUANT_NONE, WARP>, dim3(grid), dim3(threads), 0, a);
    if (a.quant == MOE_QUANT_FP8_G128)
        return launch_pdl(ctx, rmsnorm_kernel<V, MOE_QUANT_FP8_G128, WARP>, dim3(grid), dim3(threads), 0, a);
    return launch_pdl(ctx, rmsnorm_kernel<V, MOE_QUANT_FP8_G128_UE8M0, WARP>, dim3(grid), dim3(threads), 0, a);
}

template <int V, bool WARP>
cudaError_t launch_grad(const LaunchCtx& ctx, const NormGrad& a, int threads) {
    const size_t smem = WARP ? size_t(kWarpRows) * a.H * sizeof(float) : 0;
    return launch_pdl(ctx, rmsnorm_backward_kernel<V, WARP>, dim3(unsigned(norm_backward_blocks(a.T, a.H))),
                      dim3(threads), smem, a);
}

int block_threads(int H, int V) { return ((H / 8 + V - 1) / V + 31) / 32 * 32; }

}  // namespace

cudaError_t launch_rmsnorm(const LaunchCtx& ctx, const Norm& a) {
    if (a.H <= 256) return launch_norm<1, true>(ctx, a, kWarpRows * 32);
    if (a.H <= 512) return launch_norm<2, true>(ctx, a, kWarpRows * 32);
    if (a.H <= 1024) return launch_norm<4, true>(ctx, a, kWarpRows * 32);
    if (a.H <= 8192) return launch_norm<2, false>(ctx, a, block_threads(a.H, 2));
    return launch_norm<4, false>(ctx, a, block_threads(a.H, 4));
}

int norm_backward_blocks(int64_t T, int H) {
    const int64_t need = H <= 1024 ? (T + kWarpRows - 1) / kWarpRows : T;
    return int(need < kGradBlocks ? need : kGradBlocks);
}

cudaError_t launch_rmsnorm_backward(const LaunchCtx& ctx, const NormGrad& a) {
    cudaError_t err = cudaSuccess;
    if (a.T > 0) {
        if (a.H <= 256)
            err = launch_grad<1, true>(ctx, a, kWarpRows * 32);
        else if (a.H <= 512)
            err = launch_grad<2, true>(ctx, a, kWarpRows * 32);
        else if (a.H <= 1024)
            err = launch_grad<4, true>(ctx, a, kWarpRows * 32);
        else if (a.H <= 8192)
            err = launch_grad<2, false>(ctx, a, block_threads(a.H, 2));
        else
            err = launch_grad<4, false>(ctx, a, block_threads(a.H, 4));
    }
    if (err != cudaSuccess) return err;
    return launch_pdl(ctx, add_lines_kernel, dim3(unsigned((a.H + 31) / 32)), dim3(256), 0,
                      static_cast<const float*>(a.partial), norm_backward_blocks(a.T, a.H), a.H, a.grad_weight);
}

}  // namespace moe
