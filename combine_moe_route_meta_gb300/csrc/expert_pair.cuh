// expert_pair.cuh -- what the bf16 products of pairs of SMs share: the experts' row tiles, the ring's barriers, bounded
// waits, the start and the end of a kernel.
#pragma once

#include <cstdint>

#include "block_launch.h"
#include "expert_rows.cuh"
#include "tcgen05.cuh"
#include "tensor_map.h"

namespace moe {

constexpr int kPairK = 64;                                 // values of the summed index in a slot: rows of 128 bytes
constexpr uint32_t kPairBytes = 128 * 128;                 // 128 of these rows: an operand's part of a slot in one block
// Slots of a ring, at most. More of few rows get in each other's way in DRAM: 256 experts of 4 rows, 1024 -> 7168: 8 slots
// 552 us, 10 562, 12 569.
constexpr int kPairSlots = 8;
constexpr size_t kPairShared = 227 * 1024;                 // shared memory of a block, at most
constexpr int kPairEpilogueWarps = 8;
constexpr int kPairWarps = 4 + kPairEpilogueWarps;         // 0, 1: loads, products; 2: b's loads of the sums; 3: none
constexpr int kPairThreads = kPairWarps * 32;
constexpr uint32_t kPairTmemColumns = 512;                 // two accumulators of 256

struct PairShared {
    // full, acc_empty, top_empty: the leader's alone are used
    uint64_t full[kPairSlots], empty[kPairSlots], acc_full[2], acc_empty[2], top_empty[2];
    uint32_t tmem;
    int dead;   // a wait gave up
    int tiles;  // row tiles of all experts
    int most;   // rows of the largest
    // behind: prefix [E + 1], row tiles of the experts before e; base [E], first rows; count [E], rows
    __device__ __forceinline__ int* prefix() { return reinterpret_cast<int*>(this + 1); }
    __device__ __forceinline__ int* base(int E) { return prefix() + E + 1; }
    __device__ __forceinline__ int* count(int E) { return base(E) + E; }
};
constexpr size_t pair_shared_bytes(int E) { return sizeof(PairShared) + size_t(3 * E + 1) * 4; }

// A value that is the same in all lanes, as the compiler then knows.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(kFullMask, v, 0); }

// Bounded waits, which mark the block dead when they give up.
__device__ __forceinline__ bool gave_up(PairShared* s, int32_t* status) {
    *const_cast<volatile int*>(&s->dead) = 1;
    set_status(status, MOE_ERR_TIMEOUT);
    return false;
}
__device__ __forceinline__ bool pair_wait(PairShared* s, int32_t* status, uint32_t bar, uint32_t parity,
                                          uint64_t limit_ns = kWaitLimitNs) {
    return mbar_wait(bar, parity, limit_ns) || gave_up(s, status);
}
// The same for a whole warp: every lane gets the same answer.
__device__ __forceinline__ bool pair_wait_warp(PairShared* s, int32_t* status, uint32_t bar, uint32_t parity,
                                               uint64_t limit_ns = kWaitLimitNs) {
    return __all_sync(kFullMask, pair_wait(s, status, bar, parity, limit_ns));
}
// ... for a phase that threads of the other block complete too
__device__ __forceinline__ bool pair_wait_cluster(PairShared* s, int32_t* status, uint32_t bar, uint32_t parity) {
    bool done = mbar_try_wait_cluster(bar, parity);
    if (!done) {
        const uint64_t t0 = global_ns();
        int polls = 1;
        while (!(done = mbar_try_wait_cluster(bar, parity))) {
            if (polls < kWaitMinPolls)
                polls++;
            else if (global_ns() - t0 > kWaitLimitNs)
                break;
        }
    }
    return __all_sync(kFullMask, done || gave_up(s, status));
}

// True in all 128 threads of an epilogue group if it is in each of them: who gives up does not leave the others at a barrier.
__device__ __forceinline__ bool group_all(int group, bool mine) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %2, 0;\n\t"
        "barrier.cta.red.and.pred q, %1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"(1 + group), "r"(uint32_t(mine))
        : "memory");
    return all != 0;
}
__device__ __forceinline__ void group_sync(int group) {
    asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + group) : "memory");
}

// What a tile of n rows costs for each 64 values of k, in ns (measured: 277 for 192 rows, 345 for 256, 388 for 288); and what
// one of more than 256 costs besides, because its products and the next tile's cannot run beside its epilogue's start.
__device__ __forceinline__ float tile_cost(float n) { return 75.0f + 1.05f * n; }
constexpr float kWideCost = 2000.0f;
constexpr int kWideRows = 288;

// The most rows of a tile: 256, 128 or 64, whichever makes the last pair finish first, if the tiles were all alike. Small
// tiles are for few of them: 16 experts of 356 rows, dSwiGLU 2112 x 704: 29 us with 128 rows, 36 with 256.
constexpr int kRowChoices = 3;
// 256 >> the result.
__device__ __forceinline__ int pick_tile_rows(const uint32_t (&tiles)[kRowChoices], uint32_t rows, int tiles_n, int pairs) {
    int best = 0;
    float least = __int_as_float(0x7f800000);
#pragma unroll
    for (int i = 0; i < kRowChoices; i++) {
        const float rounds = __fdividef(float(tiles[i]) * float(tiles_n), float(pairs));
        if (tiles[i] == 0 || (i > 0 && rounds > 16.0f)) continue;  // many tiles: the last round hardly matters
        const float cost = ceilf(rounds) * tile_cost(__fdividef(float(rows), float(tiles[i])));
        if (cost < least) least = cost, best = i;
    }
    return best;
}
// An expert's rows in `tiles` of up to 256, or in fewer of up to 288 where k (of `chunks` times 64) is long enough: one of 280
// rows for two of 140. (256 experts of 256 +- 16 rows, SwiGLU 7168 -> 1024: 1303 us for 1420; with k = 1536 it would lose.)
__device__ __forceinline__ uint32_t wide_tiles(uint32_t rows, uint32_t tiles, int chunks) {
    const uint32_t wide = (rows + kWideRows - 1) / kWideRows;
    if (tiles < 2 || wide == tiles) return tiles;
    const float n = __fdividef(float(rows), float(tiles)), n_wide = __fdividef(float(rows), float(wide));
    return float(wide) * (tile_cost(n_wide) * chunks + kWideCost) < float(tiles) * tile_cost(n) * chunks ? wide : tiles;
}

// The start of a kernel, by all threads of both blocks: barriers (`readers`: warps of a block that read an accumulator),
// tensor memory, the experts' rows. tiles_n > 0: their row tiles too, with so many column tiles each and `chunks` slots a
// tile; experts that share rows so that there are more tiles than the output could have are refused.
__device__ __forceinline__ void pair_start(PairShared* s, const RowLayout& rows, int tiles_n, int chunks, int readers) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, E = rows.E;
    if (warp == 1) pair_tmem_alloc(smem_addr(&s->tmem), kPairTmemColumns);
    if (threadIdx.x < kPairSlots) {
        mbar_init(smem_addr(&s->full[threadIdx.x]), 1);
        mbar_init(smem_addr(&s->empty[threadIdx.x]), 1);
        if (threadIdx.x < 2) {
            mbar_init(smem_addr(&s->acc_full[threadIdx.x]), 1);
            mbar_init(smem_addr(&s->acc_empty[threadIdx.x]), 2 * readers);
            mbar_init(smem_addr(&s->top_empty[threadIdx.x]), 2 * readers);
        }
        mbar_fence_init();
    }
    if (threadIdx.x == 0) {
        s->dead = 0;
        s->tiles = 0, s->most = 0;
        s->prefix()[0] = 0;
    }
    pdl_wait();
    for (int e = threadIdx.x; e < E; e += kPairThreads) {
        const RowSpan r = expert_rows(rows, e);
        s->base(E)[e] = int(r.base);
        s->count(E)[e] = r.count;
    }
    __syncthreads();
    if (warp == 0 && tiles_n > 0) {
        uint32_t tiles[kRowChoices] = {}, all = 0, most = 0;
        for (int e = lane; e < E; e += 32) {
            const uint32_t c = s->count(E)[e];
            all += c;
            most = max(most, c);
            // kept below what 32 lanes could overflow with, and above what experts that share no row have
#pragma unroll
            for (int i = 0; i < kRowChoices; i++) tiles[i] = min(tiles[i] + ((c + (256u >> i) - 1) >> (8 - i)), 1u << 26);
        }
        all = __reduce_add_sync(kFullMask, all);
        most = __reduce_max_sync(kFullMask, most);
#pragma unroll
        for (int i = 0; i < kRowChoices; i++) tiles[i] = __reduce_add_sync(kFullMask, tiles[i]);
        // Experts that share no row have at most so many tiles, and their tiles of the output are counted in 31 bits
        // (checked on the host). Overlapping segments could have any number of both.
        if (int64_t(tiles[0]) > rows.rows / 256 + E) {
            if (lane == 0) set_status(rows.status, MOE_ERR_INVALID_ARG);
        } else {
            const int shift = 8 - pick_tile_rows(tiles, all, tiles_n, gridDim.x / 2);
            const bool wide = shift == 8 && most > 256;
            most = wide ? 0 : min(most, 1u << shift);
            int sum = 0;
            for (int e0 = 0; e0 < E; e0 += 32) {
                const uint32_t c = e0 + lane < E ? s->count(E)[e0 + lane] : 0;
                int v = int((c + (1u << shift) - 1) >> shift);
                if (wide) {
                    v = int(wide_tiles(c, v, chunks));
                    if (v > 0) most = max(most, (c + v - 1) / v);
                }
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int u = __shfl_up_sync(kFullMask, v, o);
                    if (lane >= o) v += u;
                }
                if (e0 + lane < E) s->prefix()[e0 + lane + 1] = sum + v;
                sum += __shfl_sync(kFullMask, v, 31);
            }
            if (wide) most = __reduce_max_sync(kFullMask, most);
            if (lane == 0) s->tiles = sum, s->most = int(most);
        }
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
}

// The end of a kernel, by all threads of both blocks.
__device__ __forceinline__ void pair_end(PairShared* s) {
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*const_cast<volatile int*>(&s->dead) && threadIdx.x == 0) {
        // whatever is still in flight lands in this block's memory: give it time before that is freed
        const uint64_t t0 = global_ns();
        while (global_ns() - t0 < kDrainLimitNs) __nanosleep(1000);
    }
    __syncwarp();
    cluster_sync();
    tc_fence_after();
    if (threadIdx.x / 32 == 1) pair_tmem_free(s->tmem, kPairTmemColumns);
}

// By the loading warp when it has nothing more to load, of a ring of `slots`: every product has read its slot, and no arrival
// is on its way to this block any more.
__device__ __forceinline__ void pair_drain(PairShared* s, int32_t* status, int st, uint32_t ph, int slots) {
    for (int i = 0; i < slots; i++) {
        if (!pair_wait_warp(s, status, smem_addr(&s->empty[st]), ph ^ 1)) return;
        if (++st == slots) st = 0, ph ^= 1;
    }
}

// Launches `kern` on one pair of blocks for every two SMs.
template <typename Kernel, typename... Args>
cudaError_t launch_pairs(const LaunchCtx& ctx, Kernel kern, size_t smem, Args... args) {
    const int pairs = ctx.num_sms / 2 > 0 ? ctx.num_sms / 2 : 1;
    return launch_pdl(ctx, kern, dim3(unsigned(2 * pairs)), dim3(kPairThreads), smem, args...);
}

}  // namespace moe
