// expert_wgrad_bf16.cu -- the gradient of the experts' weights: out[e, i, j] (+)= sum_r a[r, i] b[r, j] over the rows
// of each expert.
//
// Persistent pairs of SMs, each walking over tiles of 256 x 256 results of one expert: the columns of `a` are the M side of
// the products, 128 in each block, those of `b` the N side, half of them in each block (128 or 256 by what is left of n).
// Both operands are read as they lie, rows of the summed index with M or N along them, and multiplied along their columns.
// Warps have roles as in the row products; the epilogue's warps store 128 bytes of 32 rows at a time.
//
// The rows behind an expert's last belong to others, or to nobody: they may hold anything, NaNs too, and must not be summed.
// So the last slot of a tile ends with the expert's rows: these come in boxes of 32, 16, 8, 4, 2 and 1 rows as their number
// has these bits, and what is missing to 16, the step of a product, likewise in boxes that lie outside of the tensor, which
// read as zero. (128 experts of 512 +- 21 rows, 1536 x 4096 in bf16: 578 us, with boxes of 8 rows and of one alone 594.)
//
// What it measured (one GB300, single passes):
//   8 experts of 8192 rows, 4096 x 4096 in fp32:            1155 us, 1.90 PFLOP/s
//   128 experts of 512 +- 21 rows, 1536 x 4096 in fp32:     800 us, 3.2 GB of results beside 8 GB of loads from L2
//   ... in bf16:                                            579 us, 1.43 PFLOP/s
//   32 experts of one row, 1040 x 1544 in bf16:             32 us, 3.2 TB/s; without a row 21 us
#include <cstdint>

#include "expert_pair.cuh"

namespace moe {
namespace {

constexpr int kTile = 256;
constexpr uint32_t kSlot = 2 * kPairBytes;  // 64 rows of 128 columns of a, and of b
constexpr int kStages = kPairRing / kSlot;
constexpr uint32_t kStaged = 32 * 128;                              // an epilogue warp's rows on their way out
constexpr uint32_t kStaging = kPairEpilogueWarps * kStaged;         // of one buffer a warp
constexpr size_t shared_bytes(int E, int buffers) { return 1024 + kPairRing + buffers * kStaging + pair_shared_bytes(E); }
constexpr size_t kSharedMost = 227 * 1024;
static_assert(shared_bytes(MOE_MAX_EXPERTS, 1) <= kSharedMost, "shared memory of an SM");

struct GradArgs {
    WeightGrad g;
    int tiles_m, tiles_n;
    int buffers;  // of a warp: 1 or 2
};
constexpr int kBoxes = 7;
struct GradMaps {
    CUtensorMap a[kBoxes], b[kBoxes];  // boxes of 64 columns x 64, 32, .. 1 rows
};

// The tiles of a pair, one after the other: the column tiles of an expert with the row tiles of each next to each other. A
// step adds its quotients and remainders, with carries, where divisions would take a good part of a short expert's time (32
// experts of one row, 1040 x 1544: 36.6 -> 35.8 us).
struct Tiles {
    int e, m, n;             // expert, row tile, column tile
    int step_e, step_m, step_n;
    __device__ __forceinline__ Tiles(const GradArgs& a, int first, int step) {
        const int per = a.tiles_m * a.tiles_n;
        e = first / per, n = first % per / a.tiles_m, m = first % per % a.tiles_m;
        step_e = step / per, step_n = step % per / a.tiles_m, step_m = step % per % a.tiles_m;
    }
    __device__ __forceinline__ void next(const GradArgs& a) {
        m += step_m, n += step_n, e += step_e;
        if (m >= a.tiles_m) m -= a.tiles_m, n++;
        if (n >= a.tiles_n) n -= a.tiles_n, e++;
    }
};

struct Tile {
    int e, m0, n0;
    int row0, rows;  // the expert's
    int blocks;      // blocks of 64 columns of b in each of the two
    __device__ __forceinline__ Tile(const GradArgs& a, PairShared* s, const Tiles& t)
        : e(uniform(t.e)),
          m0(uniform(t.m) * kTile),
          n0(uniform(t.n) * kTile),
          row0(uniform(s->base(a.g.rows.E)[t.e])),
          rows(uniform(s->count(a.g.rows.E)[t.e])),
          blocks(a.g.n - n0 > kTile / 2 ? 2 : 1) {}
};

// A whole warp for each operand; one lane issues, with operands that are the same in all lanes (others cost 60 % more time
// for a slot).
template <bool B>
__device__ __forceinline__ void load_role(const GradArgs& a, PairShared* s, uint32_t slots, int rank,
                                          const CUtensorMap* maps) {
    const int pairs = gridDim.x / 2;
    const uint32_t own = smem_addr(s->full), counted = leaders(own), empty = smem_addr(s->empty);
    const uint32_t leader = elect_one();
    int st = 0;
    uint32_t ph = 0;
    for (Tiles t(a, blockIdx.x / 2, pairs); t.e < a.g.rows.E; t.next(a)) {
        const Tile tile(a, s, t);
        const int blocks = 2 + tile.blocks, x = B ? tile.n0 + rank * tile.blocks * 64 : tile.m0 + rank * 128;
        const bool second = !B || tile.blocks == 2;
        for (int r0 = 0; r0 < tile.rows; r0 += kPairK) {
            if (!pair_wait_warp(s, a.g.rows.status, empty + 8 * st, ph ^ 1)) return;
            if (leader) {
                const uint32_t bar = counted + 8 * st, slot = slots + st * kSlot + (B ? kPairBytes : 0);
                const int rem = min(kPairK, tile.rows - r0), row = tile.row0 + r0;
                // one box of each block of 64 columns, to rows at `to` of the slot
                const auto load = [&](int i, int to, int from) {
                    pair_load_2d(slot + to * 128, maps + i, x, from, bar);
                    if (second) pair_load_2d(slot + kPairBytes / 2 + to * 128, maps + i, x + 64, from, bar);
                };
                if (!B && rank == 0) mbar_expect_tx(own + 8 * st, 2 * blocks * ((rem + 15) & ~15) * 128);
                if (rem == kPairK) {
                    load(0, 0, row);
                } else {
                    const int gap = -rem & 15;
                    int at = 0;
                    for (int i = 1, rows = 32; i < kBoxes; i++, rows /= 2) {
                        if (rem & rows) {
                            load(i, at, row + at);
                            at += rows;
                        }
                    }
                    for (int i = 3, rows = 8; i < kBoxes; i++, rows /= 2) {
                        if (gap & rows) {
                            load(i, at, -rows);
                            at += rows;
                        }
                    }
                }
            }
            __syncwarp();
            if (++st == kStages) st = 0, ph ^= 1;
        }
    }
    if (!B) pair_drain(s, a.g.rows.status, st, ph, kStages);
}

// A whole warp of the leading block; one lane issues.
__device__ __forceinline__ void mma_role(const GradArgs& a, PairShared* s, uint32_t slots) {
    const uint64_t da = desc_mn128(slots), db = desc_mn128(slots + kPairBytes);
    const uint32_t full = smem_addr(s->full), empty = smem_addr(s->empty), tmem = uniform(s->tmem);
    const int pairs = gridDim.x / 2;
    const uint32_t leader = elect_one();
    int st = 0, n_tile = 0;
    uint32_t ph = 0;
    for (Tiles t(a, blockIdx.x / 2, pairs); t.e < a.g.rows.E; t.next(a)) {
        const Tile tile(a, s, t);
        if (tile.rows == 0) continue;
        const uint32_t idesc = pair_idesc_bf16(tile.blocks * 128, true, true);
        const int acc = n_tile & 1;
        const uint32_t d = tmem + acc * kTile;
        if (!pair_wait_cluster(s, a.g.rows.status, smem_addr(&s->acc_empty[acc]), (n_tile >> 1 & 1) ^ 1)) return;
        tc_fence_after();
        n_tile++;
        for (int r0 = 0; r0 < tile.rows; r0 += kPairK) {
            if (!pair_wait_warp(s, a.g.rows.status, full + 8 * st, ph)) return;
            tc_fence_after();
            const uint32_t off = st * (kSlot / 16);
            const int steps = (min(kPairK, tile.rows - r0) + 15) / 16;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                if (j >= steps) break;
                pair_mma_bf16(leader, d, da + off + 128 * j, db + off + 128 * j, idesc, r0 > 0 || j > 0);
            }
            pair_commit(leader, empty + 8 * st);
            if (r0 + kPairK >= tile.rows) pair_commit(leader, smem_addr(&s->acc_full[acc]));
            if (++st == kStages) st = 0, ph ^= 1;
        }
    }
}

// The sums of two columns as one word of bf16.
__device__ __forceinline__ uint32_t pack_sums(const uint32_t* r) {
    return pack_bf16x2(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Groups of four warps take tiles in turn, each an accumulator of its own: what one waits for the other's work hides, which
// counts where experts are short. A warp's 32 rows, 128 bytes of each at a time: lanes have a row each, which goes through shared memory in the 128-byte
// swizzle to a tensor store, so that whole lines reach L2 (written by the lanes themselves, 32 bytes in 32 lines at a time,
// 128 experts' 1536 x 4096 of 512 rows took 906 us). fp32 sums are added to out by the store itself.
template <bool FP32>
__device__ __forceinline__ void epilogue_role(const GradArgs& a, PairShared* s, uint32_t staging, int rank, int warp,
                                              const CUtensorMap* map_out) {
    constexpr int kCols = FP32 ? 32 : 64, kPieces = FP32 ? 2 : 2;
    const int lane = threadIdx.x % 32, quad = warp % 4, group = (warp - 4) / 4;
    const uint32_t tmem = s->tmem + (uint32_t(quad * 32) << 16);  // the 32 lanes that the warp may read
    const uint32_t first = staging + (warp - 4) * a.buffers * kStaged, other = (a.buffers - 1) * kStaged;
    uint32_t at = 0;
    const int pairs = gridDim.x / 2;
    int n_tile = 0, n_empty = 0;
    for (Tiles t(a, blockIdx.x / 2, pairs); t.e < a.g.rows.E; t.next(a)) {
        const Tile tile(a, s, t);
        const int m0 = tile.m0 + rank * 128 + quad * 32;
        const int width = m0 < a.g.m ? min(tile.blocks * 128, a.g.n - tile.n0) : 0;  // columns of the warp's rows
        const bool sums = tile.rows > 0;
        const int turn = sums ? n_tile++ : n_empty++, acc = turn & 1;
        if (acc != group || (!sums && a.g.accumulate)) continue;
        if (sums) {
            if (!pair_wait_warp(s, a.g.rows.status, smem_addr(&s->acc_full[acc]), turn >> 1 & 1)) break;
            tc_fence_after();
        }
        const auto release = [&] {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(leaders(smem_addr(&s->acc_empty[acc])));
        };
        if (sums && width == 0) release();
        // bf16: two pieces at a time, so that the accumulator is free a piece earlier
        for (int c0 = 0; c0 < width; c0 += kPieces * kCols) {
            uint32_t w[kPieces][32] = {};
#pragma unroll
            for (int i = 0; i < kPieces; i++) {
                const int c = c0 + i * kCols;
                if (!sums || c >= width) break;
                if constexpr (FP32) {
                    tmem_load32(tmem + acc * kTile + c, w[i]);
                    tmem_wait(w[i], 32);
                } else {
                    uint32_t r[64];
                    tmem_load32(tmem + acc * kTile + c, r);
                    tmem_load32(tmem + acc * kTile + c + 32, r + 32);
                    tmem_wait(r, 64);
                    if (a.g.accumulate && m0 + lane < a.g.m) {
                        const uint16_t* p = static_cast<const uint16_t*>(a.g.out) +
                                            (int64_t(tile.e) * a.g.m + m0 + lane) * a.g.n + tile.n0 + c;
#pragma unroll
                        for (int j = 0; j < 8; j++) {
                            if (tile.n0 + c + j * 8 >= a.g.n) break;
                            float x[8];
                            unpack8(*reinterpret_cast<const uint4*>(p + j * 8), x);
#pragma unroll
                            for (int l = 0; l < 8; l++)
                                r[j * 8 + l] = __float_as_uint(__uint_as_float(r[j * 8 + l]) + x[l]);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 32; j++) w[i][j] = pack_sums(r + 2 * j);
                }
            }
            if (sums && c0 + kPieces * kCols >= width) release();
#pragma unroll
            for (int i = 0; i < kPieces; i++) {
                const int c = c0 + i * kCols;
                if (c >= width) break;
                // the last store from the buffer has read it
                if (lane == 0) {
                    if (other)
                        bulk_wait_read<1>();
                    else
                        bulk_wait_read<0>();
                }
                __syncwarp();
                const uint32_t buffer = first + at, mine = buffer + lane * 128;
                at ^= other;
#pragma unroll
                for (int j = 0; j < 8; j++)
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(mine + ((j ^ (lane & 7)) << 4)),
                                 "r"(w[i][4 * j]), "r"(w[i][4 * j + 1]), "r"(w[i][4 * j + 2]), "r"(w[i][4 * j + 3])
                                 : "memory");
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
                    tma_store_3d(map_out, tile.n0 + c, m0, tile.e, buffer, FP32 && a.g.accumulate);
                    bulk_commit();
                }
                __syncwarp();
            }
        }
    }
    if (lane == 0) bulk_wait_all();
}

template <bool FP32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    weight_grad_kernel(const __grid_constant__ GradArgs a, const __grid_constant__ GradMaps maps,
                       const __grid_constant__ CUtensorMap map_out) {
    extern __shared__ uint8_t raw[];
    uint8_t* base = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);  // slots on swizzle atoms
    const uint32_t slots = smem_addr(base);
    PairShared* s = reinterpret_cast<PairShared*>(base + kPairRing + a.buffers * kStaging);
    const int warp = threadIdx.x / 32, rank = int(cluster_rank());
    pair_start(s, a.g.rows, 0, kPairEpilogueWarps / 2);
    if (warp == 0) {
        load_role<false>(a, s, slots, rank, maps.a);
    } else if (warp == 2) {
        load_role<true>(a, s, slots, rank, maps.b);
    } else if (warp == 1) {
        if (rank == 0) mma_role(a, s, slots);
    } else if (warp >= 4) {
        epilogue_role<FP32>(a, s, slots + kPairRing, rank, warp, &map_out);
    }
    pair_end(s);
}

}  // namespace

cudaError_t launch_weight_grad(const LaunchCtx& ctx, const WeightGrad& g) {
    auto kern = g.fp32 ? weight_grad_kernel<true> : weight_grad_kernel<false>;
    // first: it makes the device's context current in a thread that has made no CUDA call yet, and the maps need one
    const cudaError_t err = allow_shared_memory(kern, kSharedMost);
    if (err != cudaSuccess) return err;
    GradMaps maps{};
    CUtensorMap map_out;
    const uint64_t rows = uint64_t(g.rows.rows), da[2] = {uint64_t(g.m), rows}, db[2] = {uint64_t(g.n), rows};
    const uint64_t dout[3] = {uint64_t(g.n), uint64_t(g.m), uint64_t(g.rows.E)};
    const uint32_t bout[3] = {g.fp32 ? 32u : 64u, 32, 1};
    for (int i = 0; i < kBoxes && rows > 0; i++) {  // without rows nothing is loaded
        const uint32_t box[2] = {64, uint32_t(kPairK) >> i};
        if (!make_map_bf16(&maps.a[i], g.a, 2, da, box) || !make_map_bf16(&maps.b[i], g.b, 2, db, box))
            return cudaErrorInvalidValue;
    }
    if (!(g.fp32 ? make_map_fp32(&map_out, g.out, 3, dout, bout) : make_map_bf16(&map_out, g.out, 3, dout, bout)))
        return cudaErrorInvalidValue;
    const int buffers = shared_bytes(g.rows.E, 2) <= kSharedMost ? 2 : 1;
    const GradArgs a{g, (g.m + kTile - 1) / kTile, (g.n + kTile - 1) / kTile, buffers};
    return launch_pairs(ctx, kern, shared_bytes(g.rows.E, buffers), a, maps, map_out);
}

}  // namespace moe
