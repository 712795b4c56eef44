// rmsnorm.cu -- root-mean-square norm of x + residual, in bf16 and in FP8 with a scale for each 128 values, and its
// gradient.
//
// A row stays in registers between its one reading and its one writing. A lane has runs of 8 columns, threads next to
// each other neighbouring runs, so accesses are of 16 bytes and the 128 values of an FP8 group lie in 16 neighbouring
// lanes. Rows of up to 1024 columns are a warp's, longer ones a block's. As many blocks as fit go from row to row, with the
// next row's loads on their way beside this one's reduction; large gradients have up to four rows ahead in shared memory. The
// gradient of the weight is a sum over rows: each of at most kGradBlocks blocks sums its rows in registers and writes one line
// of partial sums; a second kernel adds the lines in order.
//
// Bound by DRAM; one GB300, whose copy bandwidth is 6777 GB/s, cold L2:
//   16384 x 4096, residual:  FP8 72 us (6.5 TB/s), bf16 87 us (6.1), gradient 82 us (6.6)
//   8192 x 7168:             FP8 64 us (6.4 TB/s), bf16 76 us (6.1), gradient 77 us (6.1)
//   128 x 7168:              FP8 2.8 us, bf16 2.3 us, gradient 5.7 us (two launches)
// One row a block, and no loads ahead: 100, 97 and 147 us for the first.
#include <cstdint>

#include "block_launch.h"
#include "dispatch_slice.cuh"
#include "moe_block.h"
#include "moe_device.cuh"

namespace moe {
namespace {

constexpr int kGradBlocks = 304;
constexpr int64_t kManyValues = 1 << 24;
constexpr size_t kRowsAhead = 108 * 1024;  // shared memory for rows on their way, for two blocks on an SM
constexpr int kWarpColumns = 1024;  // of a warp's row, at most
// Warps of a block with a row each: the gradient's blocks are few, so they have more warps where registers allow.
template <int V, bool GRAD>
constexpr int kWarpRows = GRAD && V < 4 ? 16 / V : 4;
// Whether a row is loaded beside the one before and the weight stays in registers: not in the gradient's blocks with four runs
// of columns a thread, nor in blocks of up to 1024 threads.
template <int V, bool WARP, int THREADS, bool GRAD>
constexpr bool kAhead = WARP || V < 4 || (THREADS == 512 && !GRAD);

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

// Where a thread's rows and columns lie: a warp's rows go from warp to warp of the grid, a block's from block to block.
template <bool WARP>
struct Place {
    int lane, lanes;
    int64_t first, step;
    __device__ __forceinline__ Place()
        : lane(WARP ? threadIdx.x % 32 : threadIdx.x),
          lanes(WARP ? 32 : blockDim.x),
          first(WARP ? (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) / 32 : blockIdx.x),
          step(WARP ? int64_t(gridDim.x) * (blockDim.x / 32) : gridDim.x) {}
    __device__ __forceinline__ int column(int v) const { return (v * lanes + lane) * 8; }
};

// A thread's part of a row, zeros beyond its end; all zeros for p null.
template <int V, bool WARP>
__device__ __forceinline__ void load_row(uint4 (&r)[V], const uint16_t* p, int64_t t, int H, const Place<WARP>& at) {
#pragma unroll
    for (int v = 0; v < V; v++)
        r[v] = p && at.column(v) < H ? ld_v4(p + t * H + at.column(v)) : make_uint4(0, 0, 0, 0);
}

template <int V, int QUANT, bool WARP, int THREADS>
__global__ void __launch_bounds__(THREADS) rmsnorm_kernel(Norm a) {
    __shared__ float part[2][32];
    pdl_wait();
    const Place<WARP> at;
    uint4 w[V], x[V], res[V];
    if (kAhead<V, WARP, THREADS, false>) load_row(w, a.weight, 0, a.H, at);
    if (kAhead<V, WARP, THREADS, false> && at.first < a.T) {
        load_row(x, a.x, at.first, a.H, at);
        load_row(res, a.residual, at.first, a.H, at);
    }
    int turn = 0;
    for (int64_t t = at.first; t < a.T; t += at.step, turn ^= 1) {
        const int64_t row = t * a.H;
        float s[V][8], square = 0.0f;
        if (!kAhead<V, WARP, THREADS, false>) {
            load_row(x, a.x, t, a.H, at);
            load_row(res, a.residual, t, a.H, at);
        }
#pragma unroll
        for (int v = 0; v < V; v++) {
            unpack8(x[v], s[v]);
            if (a.residual) {
                float r[8];
                unpack8(res[v], r);
#pragma unroll
                for (int j = 0; j < 8; j++) s[v][j] += r[j];
                // the norm is of the sum as it is stored, rounded: what the next layer and the gradient see
                const uint4 sum = pack8(s[v]);
                unpack8(sum, s[v]);
                if (a.sum && at.column(v) < a.H) st_v4(a.sum + row + at.column(v), sum);
            }
#pragma unroll
            for (int j = 0; j < 8; j++) square = fmaf(s[v][j], s[v][j], square);
        }
        if (!kAhead<V, WARP, THREADS, false>) {
            load_row(w, a.weight, 0, a.H, at);
        } else if (t + at.step < a.T) {  // the next row, beside this one's reduction
            load_row(x, a.x, t + at.step, a.H, at);
            load_row(res, a.residual, t + at.step, a.H, at);
        }
        square = row_sum<WARP>(square, part, turn);
        const float r = __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(square, float(a.H)), a.eps)));
        if (a.rstd && at.lane == 0) a.rstd[t] = r;
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int c = at.column(v);
            const bool in = c < a.H;
            float y[8];
            unpack8(w[v], y);
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
                    if (in && at.lane % 16 == 0) static_cast<float*>(a.scales)[t * (a.H / 128) + c / 128] = sc;
                } else {
                    const uint32_t bits = __float_as_uint(sc);
                    const uint32_t ex = (bits >> 23) + ((bits & 0x7fffffu) ? 1u : 0u);
                    const float inv = __uint_as_float((254u - ex) << 23);  // of a power of two: exact
#pragma unroll
                    for (int j = 0; j < 8; j++) y[j] = __fmul_rn(y[j], inv);
                    if (in && at.lane % 16 == 0) static_cast<uint8_t*>(a.scales)[t * (a.H / 128) + c / 128] = uint8_t(ex);
                }
#pragma unroll
                for (int j = 0; j < 2; j++)
                    q[j] = e4m3x2(y[4 * j], y[4 * j + 1]) | e4m3x2(y[4 * j + 2], y[4 * j + 3]) << 16;
                if (in) st_v2(a.codes + row + c, make_uint2(q[0], q[1]));
            }
        }
    }
}

template <int V, bool WARP, int THREADS>
__global__ void __launch_bounds__(THREADS) rmsnorm_backward_kernel(NormGrad a) {
    __shared__ float part[2][32];
    extern __shared__ float lines[];  // WARP: [warps][H]
    pdl_wait();
    const Place<WARP> at;
    uint4 w[V], s[V], g[V], more[V];
    float acc[V][8] = {}, r = 0.0f;
    if (kAhead<V, WARP, THREADS, true>) load_row(w, a.weight, 0, a.H, at);
    if (kAhead<V, WARP, THREADS, true> && at.first < a.T) {
        load_row(s, a.s, at.first, a.H, at);
        load_row(g, a.grad, at.first, a.H, at);
        load_row(more, a.grad_sum, at.first, a.H, at);
        r = __ldg(a.rstd + at.first);
    }
    int turn = 0;
    for (int64_t t = at.first; t < a.T; t += at.step, turn ^= 1) {
        float hat[V][8], gw[V][8], dot = 0.0f;
        uint4 add[V];
        if (!kAhead<V, WARP, THREADS, true>) {
            load_row(w, a.weight, 0, a.H, at);
            load_row(s, a.s, t, a.H, at);
            load_row(g, a.grad, t, a.H, at);
            r = __ldg(a.rstd + t);
        }
        const float r_now = r;
#pragma unroll
        for (int v = 0; v < V; v++) {
            float wv[8];
            unpack8(s[v], hat[v]);
            unpack8(g[v], gw[v]);
            unpack8(w[v], wv);
            add[v] = more[v];
#pragma unroll
            for (int j = 0; j < 8; j++) {
                hat[v][j] *= r_now;
                acc[v][j] = fmaf(gw[v][j], hat[v][j], acc[v][j]);
                gw[v][j] *= wv[j];
                dot = fmaf(gw[v][j], hat[v][j], dot);
            }
        }
        if (!kAhead<V, WARP, THREADS, true>) {
            load_row(add, a.grad_sum, t, a.H, at);
        } else if (t + at.step < a.T) {  // the next row, beside this one's reduction
            load_row(s, a.s, t + at.step, a.H, at);
            load_row(g, a.grad, t + at.step, a.H, at);
            load_row(more, a.grad_sum, t + at.step, a.H, at);
            r = __ldg(a.rstd + t + at.step);
        }
        const float mean = __fdiv_rn(row_sum<WARP>(dot, part, turn), float(a.H));
#pragma unroll
        for (int v = 0; v < V; v++) {
            if (at.column(v) >= a.H) continue;
            float d[8], f[8];
            unpack8(add[v], f);
#pragma unroll
            for (int j = 0; j < 8; j++) d[j] = fmaf(r_now, fmaf(-mean, hat[v][j], gw[v][j]), f[j]);
            st_v4(a.grad_x + t * a.H + at.column(v), pack8(d));
        }
    }
    float* line = a.partial + int64_t(blockIdx.x) * a.H;
    if constexpr (WARP) {
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int c = at.column(v);
            if (c >= a.H) continue;
#pragma unroll
            for (int j = 0; j < 8; j++) lines[threadIdx.x / 32 * a.H + c + j] = acc[v][j];
        }
        __syncthreads();
        for (int c = threadIdx.x; c < a.H; c += blockDim.x) {
            float sum = 0.0f;
            for (int i = 0; i < THREADS / 32; i++) sum += lines[i * a.H + c];
            line[c] = sum;
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; v++) {
            const int c = at.column(v);
            if (c >= a.H) continue;
            *reinterpret_cast<float4*>(line + c) = make_float4(acc[v][0], acc[v][1], acc[v][2], acc[v][3]);
            *reinterpret_cast<float4*>(line + c + 4) = make_float4(acc[v][4], acc[v][5], acc[v][6], acc[v][7]);
        }
    }
}

// A thread's parts of the next rows of N tensors, on their way to its own places in shared memory: `stages` rows ahead, without
// registers, and without a barrier since nobody else reads them. A tensor may be null: zeros.
template <int V, int N>
struct RowsAhead {
    uint32_t mine;  // this thread's place of the first run
    int stages, st = 0;
    const uint16_t* from[N];
    __device__ __forceinline__ uint32_t place(int x, int v) const {
        return mine + uint32_t(((st * N + x) * V + v) * blockDim.x) * 16;
    }
    // The part of row t into the current stage; nothing beyond the last row.
    __device__ __forceinline__ void load(int64_t t, int64_t T, int H, const Place<false>& at) {
        if (t < T) {
#pragma unroll
            for (int x = 0; x < N; x++)
#pragma unroll
                for (int v = 0; v < V; v++)
                    if (from[x] && at.column(v) < H)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(place(x, v)),
                                     "l"(from[x] + t * H + at.column(v))
                                     : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (++st == stages) st = 0;
    }
    __device__ __forceinline__ void start(int64_t T, int H, const Place<false>& at) {
        for (int i = 0; i < stages; i++) load(at.first + i * at.step, T, H, at);
    }
    // The oldest row, which lies in the current stage. The next load() comes after a barrier: the stage has been read then.
    __device__ __forceinline__ void take(uint4 (&r)[N][V], int H, const Place<false>& at) {
        if (stages == 4)
            asm volatile("cp.async.wait_group 3;" ::: "memory");
        else
            asm volatile("cp.async.wait_group 1;" ::: "memory");
#pragma unroll
        for (int x = 0; x < N; x++)
#pragma unroll
            for (int v = 0; v < V; v++) {
                r[x][v] = make_uint4(0, 0, 0, 0);
                if (from[x] && at.column(v) < H)
                    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                 : "=r"(r[x][v].x), "=r"(r[x][v].y), "=r"(r[x][v].z), "=r"(r[x][v].w)
                                 : "r"(place(x, v))
                                 : "memory");
            }
    }
};

// The same of rows of a block, with the rows ahead in shared memory.
template <int V>
__global__ void __launch_bounds__(512) rmsnorm_backward_ahead_kernel(NormGrad a, int stages) {
    __shared__ float part[2][32];
    extern __shared__ float4 rows[];
    pdl_wait();
    const Place<false> at;
    uint4 w[V];
    float acc[V][8] = {};
    load_row(w, a.weight, 0, a.H, at);
    RowsAhead<V, 3> ahead{smem_addr(rows) + threadIdx.x * 16, stages, 0, {a.s, a.grad, a.grad_sum}};
    ahead.start(a.T, a.H, at);
    float next = at.first < a.T ? __ldg(a.rstd + at.first) : 0.0f;
    int turn = 0;
    for (int64_t t = at.first; t < a.T; t += at.step, turn ^= 1) {
        uint4 row[3][V];
        ahead.take(row, a.H, at);
        const float r = next;
        if (t + at.step < a.T) next = __ldg(a.rstd + t + at.step);
        float hat[V][8], gw[V][8], dot = 0.0f;
#pragma unroll
        for (int v = 0; v < V; v++) {
            float wv[8];
            unpack8(row[0][v], hat[v]);
            unpack8(row[1][v], gw[v]);
            unpack8(w[v], wv);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                hat[v][j] *= r;
                acc[v][j] = fmaf(gw[v][j], hat[v][j], acc[v][j]);
                gw[v][j] *= wv[j];
                dot = fmaf(gw[v][j], hat[v][j], dot);
            }
        }
        const float mean = __fdiv_rn(row_sum<false>(dot, part, turn), float(a.H));
        ahead.load(t + stages * at.step, a.T, a.H, at);
#pragma unroll
        for (int v = 0; v < V; v++) {
            if (at.column(v) >= a.H) continue;
            float d[8], f[8];
            unpack8(row[2][v], f);
#pragma unroll
            for (int j = 0; j < 8; j++) d[j] = fmaf(r, fmaf(-mean, hat[v][j], gw[v][j]), f[j]);
            st_v4(a.grad_x + t * a.H + at.column(v), pack8(d));
        }
    }
    float* line = a.partial + int64_t(blockIdx.x) * a.H;
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int c = at.column(v);
        if (c >= a.H) continue;
        *reinterpret_cast<float4*>(line + c) = make_float4(acc[v][0], acc[v][1], acc[v][2], acc[v][3]);
        *reinterpret_cast<float4*>(line + c + 4) = make_float4(acc[v][4], acc[v][5], acc[v][6], acc[v][7]);
    }
}

// grad_weight[c] = the sum of `n` lines: up to 32 threads a column, each every 32nd line, then these in order.
constexpr int kParts = 32;
__global__ void __launch_bounds__(32 * kParts) add_lines_kernel(const float* lines, int n, int H, float* out) {
    __shared__ float sums[kParts][32];
    pdl_wait();
    const int c = blockIdx.x * 32 + threadIdx.x % 32, part = threadIdx.x / 32;
    float s = 0.0f;
    if (c < H) {
#pragma unroll
        for (int i = 0; i < (kGradBlocks + kParts - 1) / kParts; i++)
            if (part + i * kParts < n) s += lines[int64_t(part + i * kParts) * H + c];
    }
    sums[part][threadIdx.x % 32] = s;
    __syncthreads();
    if (part != 0 || c >= H) return;
    for (int i = 1; i < int(blockDim.x) / 32; i++) s += sums[i][threadIdx.x];
    out[c] = s;
}

template <typename Kernel>
cudaError_t launch_rows(const LaunchCtx& ctx, Kernel kern, const Norm& a, int rows, int threads) {
    int per_sm = 0;
    const cudaError_t err = blocks_per_sm(ctx, kern, threads, 0, &per_sm);
    if (err != cudaSuccess) return err;
    const int64_t need = (a.T + rows - 1) / rows;
    const int64_t most = int64_t(ctx.num_sms) * (per_sm > 0 ? per_sm : 1);
    return launch_pdl(ctx, kern, dim3(unsigned(need < most ? need : most)), dim3(threads), 0, a);
}

template <int V, bool WARP, int THREADS>
cudaError_t launch_norm(const LaunchCtx& ctx, const Norm& a, int threads) {
    const int rows = WARP ? threads / 32 : 1;
    if (a.quant == MOE_QUANT_NONE)
        return launch_rows(ctx, rmsnorm_kernel<V, MOE_QUANT_NONE, WARP, THREADS>, a, rows, threads);
    if (a.quant == MOE_QUANT_FP8_G128)
        return launch_rows(ctx, rmsnorm_kernel<V, MOE_QUANT_FP8_G128, WARP, THREADS>, a, rows, threads);
    return launch_rows(ctx, rmsnorm_kernel<V, MOE_QUANT_FP8_G128_UE8M0, WARP, THREADS>, a, rows, threads);
}
template <int V>
cudaError_t launch_norm_warps(const LaunchCtx& ctx, const Norm& a) {
    return launch_norm<V, true, kWarpRows<V, false> * 32>(ctx, a, kWarpRows<V, false> * 32);
}

template <int V, bool WARP, int THREADS>
cudaError_t launch_grad(const LaunchCtx& ctx, const NormGrad& a, int threads) {
    const size_t smem = WARP ? size_t(threads / 32) * a.H * sizeof(float) : 0;
    return launch_pdl(ctx, rmsnorm_backward_kernel<V, WARP, THREADS>, dim3(unsigned(norm_backward_blocks(a.T, a.H))),
                      dim3(threads), smem, a);
}
// Rows ahead in shared memory, four of them where two blocks on an SM have room: from 16 M values on, of up to 8192 columns.
// (16384 x 4096 82 us, by registers 90.5; 8192 x 7168 77 and 89.5; 2432 x 7168 29.6 and 32.2; 1800 x 4096 16.0 and 15.1.
// The norm itself has registers for more blocks, and loses: 16384 x 4096 in bf16 92 us for 87.)
template <int V>
cudaError_t launch_grad_ahead(const LaunchCtx& ctx, const NormGrad& a, int threads) {
    const int64_t blocks = norm_backward_blocks(a.T, a.H);
    if (a.T * a.H < kManyValues) return launch_grad<V, false, 512>(ctx, a, threads);
    auto kern = rmsnorm_backward_ahead_kernel<V>;
    const size_t row = size_t(3) * V * 16 * threads;
    const int stages = row * 4 <= kRowsAhead ? 4 : 2;
    const cudaError_t err = allow_shared_memory(kern, kRowsAhead);
    if (err != cudaSuccess) return err;
    return launch_pdl(ctx, kern, dim3(unsigned(blocks)), dim3(threads), stages * row, a, stages);
}
template <int V>
cudaError_t launch_grad_warps(const LaunchCtx& ctx, const NormGrad& a) {
    return launch_grad<V, true, kWarpRows<V, true> * 32>(ctx, a, kWarpRows<V, true> * 32);
}

// Runs of 8 columns in a thread of a block that has a row: two, one where that would leave few threads to a block (1003 rows
// of 2176: 4.5 us with one, 5.0 with two; 16384 rows of 4096 in FP8: 79 and 72 us), four beyond 512 threads.
int block_runs(int H) { return H < 4096 ? 1 : H <= 8192 ? 2 : 4; }
int block_threads(int H, int V) { return ((H / 8 + V - 1) / V + 31) / 32 * 32; }

}  // namespace

cudaError_t launch_rmsnorm(const LaunchCtx& ctx, const Norm& a) {
    if (a.H <= kWarpColumns / 4) return launch_norm_warps<1>(ctx, a);
    if (a.H <= kWarpColumns / 2) return launch_norm_warps<2>(ctx, a);
    if (a.H <= kWarpColumns) return launch_norm_warps<4>(ctx, a);
    const int V = block_runs(a.H), threads = block_threads(a.H, V);
    if (V == 1) return launch_norm<1, false, 512>(ctx, a, threads);
    if (V == 2) return launch_norm<2, false, 512>(ctx, a, threads);
    // blocks of 384 to 512 threads have registers for a row ahead (4096 x 16384: FP8 86 -> 75.5 us, bf16 88.5 -> 86); with 320,
    // three blocks without are better than one with (8192 x 10240: FP8 107 and 122 us, bf16 111 and 108)
    if (threads >= 384 && threads <= 512) return launch_norm<4, false, 512>(ctx, a, threads);
    return launch_norm<4, false, 1024>(ctx, a, threads);
}

int norm_backward_blocks(int64_t T, int H) {
    const int rows = H <= kWarpColumns / 4   ? kWarpRows<1, true>
                     : H <= kWarpColumns / 2 ? kWarpRows<2, true>
                     : H <= kWarpColumns     ? kWarpRows<4, true>
                                             : 1;
    const int64_t need = (T + rows - 1) / rows;
    return int(need < kGradBlocks ? need : kGradBlocks);
}

cudaError_t launch_rmsnorm_backward(const LaunchCtx& ctx, const NormGrad& a) {
    cudaError_t err = cudaSuccess;
    if (a.T > 0) {
        const int V = block_runs(a.H), threads = block_threads(a.H, V);
        if (a.H <= kWarpColumns / 4)
            err = launch_grad_warps<1>(ctx, a);
        else if (a.H <= kWarpColumns / 2)
            err = launch_grad_warps<2>(ctx, a);
        else if (a.H <= kWarpColumns)
            err = launch_grad_warps<4>(ctx, a);
        else if (V == 1)
            err = launch_grad_ahead<1>(ctx, a, threads);
        else if (V == 2)
            err = launch_grad_ahead<2>(ctx, a, threads);
        else if (threads <= 512)
            err = launch_grad<4, false, 512>(ctx, a, threads);
        else
            err = launch_grad<4, false, 1024>(ctx, a, threads);
    }
    if (err != cudaSuccess) return err;
    const int lines = norm_backward_blocks(a.T, a.H), parts = lines < 1 ? 1 : lines < kParts ? lines : kParts;
    return launch_pdl(ctx, add_lines_kernel, dim3(unsigned((a.H + 31) / 32)), dim3(32 * parts), 0,
                      static_cast<const float*>(a.partial), lines, a.H, a.grad_weight);
}

}  // namespace moe
