// expert_wgrad_bf16.cu -- the gradient of the experts' weights: out[e, i, j] (+)= sum_r a[r, i] b[r, j] over the rows
// of each expert.
//
// Persistent pairs of SMs, each walking over tiles of 256 x 256 results of one expert: one operand's columns are the M side
// of the products, 128 in each block, the other's the N side, half of them in each block (128 or 256 by what is left). Both
// operands are read as they lie, rows of the summed index with M or N along them, and multiplied along their columns. Warps
// have roles as in the row products, with a warp for the loads of each operand (one for both: 128 ragged experts 778 us for
// 750). Tiles that lie beside each other in the result's rows follow one another (below each other: 700 -> 715 us, in bf16
// 563 -> 578).
//
// The M side lies along the lanes of the accumulator. For fp32 results these are the columns of out: a warp stores 128
// bytes of a row, whole lines, from its registers. In bf16 that would be 64 bytes (32 experts of one row 34 us for 25): there
// the lanes are rows of out, which go through shared memory to tensor stores of 128 bytes of 32 rows.
//
// The rows behind an expert's last belong to others, or to nobody: they may hold anything, NaNs too, and must not be summed.
// So the last slot of a tile ends with the expert's rows: these come in boxes of 32, 16, 8, 4, 2 and 1 rows as their number
// has these bits, and what is missing to 16, the step of a product, likewise in boxes that lie outside of the tensor, which
// read as zero. (128 experts of 512 +- 21 rows, 1536 x 4096 in bf16: 578 us, with boxes of 8 rows and of one alone 594.)
//
// What it measured (one GB300, single passes):
//   8 experts of 8192 rows, 4096 x 4096 in fp32:            1150 us, 1.91 PFLOP/s
//   128 experts of 512 +- 21 rows, 1536 x 4096 in fp32:     695 us: 3.2 GB of results beside 8 GB of loads from L2
//   ... in bf16:                                            533 us, 1.55 PFLOP/s
//   32 experts of one row, 1040 x 1544 in bf16:             24 us, 4.3 TB/s; without a row 19.5 us
#include <cstdint>

#include "expert_pair.cuh"

namespace moe {
namespace {

constexpr int kTile = 256;
constexpr uint32_t kSlot = 2 * kPairBytes;  // 64 rows of 128 columns of each operand
constexpr uint32_t kStaged = 32 * 128;      // bf16: an epilogue warp's rows on their way out
constexpr uint32_t kStaging = kPairEpilogueWarps * kStaged;
// A group of epilogue warps waits for up to two sums, the other group's and its own next one. A slot takes 345 ns, and up to
// 600 at the 1.2 of 2.07 GHz that the power limit can leave.
constexpr uint64_t kMostSlotNs = 600;
constexpr uint64_t kSumsLimitNs = 2 * kWaitLimitNs;
static_assert(2 * (kMostSummedRows / kPairK) * kMostSlotNs <= kSumsLimitNs, "two of the longest sums end within a wait");
template <typename T>
constexpr bool kFp32 = sizeof(T) == 4;
template <typename T>
constexpr size_t shared_bytes(int slots, int E) {
    return 1024 + slots * kSlot + (kFp32<T> ? 0 : kStaging) + pair_shared_bytes(E);
}
static_assert(shared_bytes<float>(6, MOE_MAX_EXPERTS) <= kPairShared, "shared memory of an SM");
static_assert(shared_bytes<uint16_t>(5, MOE_MAX_EXPERTS) <= kPairShared, "shared memory of an SM");

struct GradArgs {
    WeightGrad g;  // a: the M side, of m columns; b: the N side, of n
    int tiles_m, tiles_n;
    int slots;
};
constexpr int kBoxes = 7;
struct GradMaps {
    CUtensorMap a[kBoxes], b[kBoxes];  // boxes of 64 columns x 64, 32, .. 1 rows
};

// The tiles of a pair, one after the other: those beside each other in out first. A step adds its quotients and remainders,
// with carries, where divisions would take a good part of a short expert's time (32 experts of one row, 1040 x 1544:
// 36.6 -> 35.8 us).
template <typename T>
struct Tiles {
    int e, row, column;  // of out
    int rows, columns;   // tiles
    int step_e, step_row, step_column;
    __device__ __forceinline__ Tiles(const GradArgs& a, int first, int step)
        : rows(kFp32<T> ? a.tiles_n : a.tiles_m), columns(kFp32<T> ? a.tiles_m : a.tiles_n) {
        const int per = rows * columns;
        e = first / per, row = first % per / columns, column = first % per % columns;
        step_e = step / per, step_row = step % per / columns, step_column = step % per % columns;
    }
    __device__ __forceinline__ void next() {
        column += step_column, row += step_row, e += step_e;
        if (column >= columns) column -= columns, row++;
        if (row >= rows) row -= rows, e++;
    }
    __device__ __forceinline__ int m() const { return kFp32<T> ? column : row; }
    __device__ __forceinline__ int n() const { return kFp32<T> ? row : column; }
};

struct Tile {
    int e, m0, n0;
    int row0, rows;  // the expert's
    int blocks;      // blocks of 64 columns of b in each of the two
    template <typename T>
    __device__ __forceinline__ Tile(const GradArgs& a, PairShared* s, const Tiles<T>& t)
        : e(uniform(t.e)),
          m0(uniform(t.m()) * kTile),
          n0(uniform(t.n()) * kTile),
          row0(uniform(s->base(a.g.rows.E)[t.e])),
          rows(uniform(s->count(a.g.rows.E)[t.e])),
          blocks(a.g.n - n0 > kTile / 2 ? 2 : 1) {}
};

// A whole warp for each operand; one lane issues, with operands that are the same in all lanes (others cost 60 % more time
// for a slot).
template <typename T, bool B>
__device__ __forceinline__ void load_role(const GradArgs& a, PairShared* s, uint32_t slots, int rank,
                                          const CUtensorMap* maps) {
    const int pairs = gridDim.x / 2;
    const uint32_t own = smem_addr(s->full), counted = leaders(own), empty = smem_addr(s->empty);
    const uint32_t leader = elect_one();
    int st = 0;
    uint32_t ph = 0;
    for (Tiles<T> t(a, blockIdx.x / 2, pairs); t.e < a.g.rows.E; t.next()) {
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
            if (++st == a.slots) st = 0, ph ^= 1;
        }
    }
    if (!B) pair_drain(s, a.g.rows.status, st, ph, a.slots);
}

// A whole warp of the leading block; one lane issues.
template <typename T>
__device__ __forceinline__ void mma_role(const GradArgs& a, PairShared* s, uint32_t slots) {
    const uint64_t da = desc_mn128(slots), db = desc_mn128(slots + kPairBytes);
    const uint32_t full = smem_addr(s->full), empty = smem_addr(s->empty), tmem = uniform(s->tmem);
    const int pairs = gridDim.x / 2;
    const uint32_t leader = elect_one();
    int st = 0, n_tile = 0;
    uint32_t ph = 0;
    for (Tiles<T> t(a, blockIdx.x / 2, pairs); t.e < a.g.rows.E; t.next()) {
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
            if (++st == a.slots) st = 0, ph ^= 1;
        }
    }
}

// What both types' epilogues walk over: groups of four warps take tiles in turn, each an accumulator of its own. What one
// waits for the other's work hides, which counts where experts are short.
struct EpilogueWarp {
    PairShared* s;
    int lane, group;
    uint32_t tmem;      // the 32 lanes that the warp may read
    int first;          // of its lanes, among the 256 of a tile
    int n_tile = 0, n_empty = 0;
    int acc = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ EpilogueWarp(PairShared* s, int rank, int warp)
        : s(s),
          lane(threadIdx.x % 32),
          group((warp - 4) / 4),
          tmem(s->tmem + (uint32_t(warp % 4 * 32) << 16)),
          first(rank * 128 + warp % 4 * 32) {}
    // Whether the next tile is the group's; a tile without rows has no accumulator.
    __device__ __forceinline__ bool takes(bool sums) {
        const int turn = sums ? n_tile++ : n_empty++;
        acc = turn & 1, phase = turn >> 1 & 1;
        return acc == group;
    }
    __device__ __forceinline__ bool wait(int32_t* status) const {
        if (!pair_wait_warp(s, status, smem_addr(&s->acc_full[acc]), phase, kSumsLimitNs)) return false;
        tc_fence_after();
        return true;
    }
    __device__ __forceinline__ uint32_t columns(int c) const { return tmem + acc * kTile + c; }
    // The accumulator has been read.
    __device__ __forceinline__ void release() const {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(leaders(smem_addr(&s->acc_empty[acc])));
    }
};

// A lane's column of up to 32 rows, from p and the rows behind it, or to them. No test stands between whole pieces' accesses:
// with one at each store, 128 experts take 1080 us for 700.
__device__ __forceinline__ void get_column(float (&r)[32], const float* p, int64_t stride, int rows) {
    if (rows >= 32) {
#pragma unroll
        for (int i = 0; i < 32; i++) r[i] = p[i * stride];
    } else {
#pragma unroll
        for (int i = 0; i < 32; i++) r[i] = i < rows ? p[i * stride] : 0.0f;
    }
}
__device__ __forceinline__ void put_column(float* p, int64_t stride, const float (&r)[32], int rows) {
    if (rows >= 32) {
#pragma unroll
        for (int i = 0; i < 32; i++) p[i * stride] = r[i];
    } else {
#pragma unroll
        for (int i = 0; i < 32; i++)
            if (i < rows) p[i * stride] = r[i];
    }
}
// An expert without rows: zeros to `rows` rows of up to 512 bytes, whole ones by a warp. (32 experts without a row, 1040 x 1544
// in fp32: 35 us, 38 by 128 bytes at a time.)
template <typename T>
__device__ __forceinline__ void put_zeros(T* p, int64_t stride, int rows, int columns, int quad, int lane) {
    const int c = lane * int(16 / sizeof(T));
    if (c >= columns) return;
#pragma unroll 8
    for (int r = quad; r < rows; r += 4) st_v4(p + r * stride + c, make_uint4(0, 0, 0, 0));
}

// Lanes are columns of out.
template <bool ADD>
__device__ __forceinline__ void epilogue_fp32(const GradArgs& a, PairShared* s, int rank, int warp) {
    EpilogueWarp me(s, rank, warp);
    const int64_t stride = a.g.m;
    for (Tiles<float> t(a, blockIdx.x / 2, gridDim.x / 2); t.e < a.g.rows.E; t.next()) {
        const Tile tile(a, s, t);
        const bool sums = tile.rows > 0;
        if (!me.takes(sums) || (!sums && ADD)) continue;
        if (!sums) {
            const int c0 = tile.m0 + rank * 128;
            put_zeros(static_cast<float*>(a.g.out) + (int64_t(tile.e) * a.g.n + tile.n0) * stride + c0, stride,
                      min(tile.blocks * 128, a.g.n - tile.n0), a.g.m - c0, warp % 4, me.lane);
            __syncwarp();
            continue;
        }
        const int column = tile.m0 + me.first + me.lane;
        const int rows = tile.m0 + me.first < a.g.m ? min(tile.blocks * 128, a.g.n - tile.n0) : 0;
        const int mine = column < a.g.m ? rows : 0;
        float* p = static_cast<float*>(a.g.out) + (int64_t(tile.e) * a.g.n + tile.n0) * stride + column;
        float old[32];
        if (ADD) get_column(old, p, stride, mine);
        if (!me.wait(a.g.rows.status)) break;
        if (rows == 0) me.release();
        for (int c = 0; c < rows; c += 32, p += 32 * stride) {
            uint32_t w[32];
            tmem_load32(me.columns(c), w);
            tmem_wait(w, 32);
            if (c + 32 >= rows) me.release();
            float r[32];
#pragma unroll
            for (int i = 0; i < 32; i++) r[i] = __uint_as_float(w[i]);
            if (ADD) {
#pragma unroll
                for (int i = 0; i < 32; i++) r[i] += old[i];
                if (c + 32 < rows) get_column(old, p + 32 * stride, stride, mine - c - 32);
            }
            put_column(p, stride, r, mine - c);
            __syncwarp();
        }
    }
}

// The sums of two columns as one word of bf16.
__device__ __forceinline__ uint32_t pack_sums(const uint32_t* r) {
    return pack_bf16x2(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Lanes are rows of out. A warp's 32 rows, 128 bytes of each at a time, go through shared memory in the 128-byte swizzle to
// a tensor store. Two pieces are taken before they are written, so that the accumulator is free a piece earlier (32 experts
// of one row 31.5 -> 29.4 us).
template <bool ADD>
__device__ __forceinline__ void epilogue_bf16(const GradArgs& a, PairShared* s, uint32_t staging, int rank, int warp,
                                              const CUtensorMap* map_out) {
    constexpr int kCols = 64, kPieces = 2;
    EpilogueWarp me(s, rank, warp);
    const uint32_t buffer = staging + (warp - 4) * kStaged, mine = buffer + me.lane * 128;
    for (Tiles<uint16_t> t(a, blockIdx.x / 2, gridDim.x / 2); t.e < a.g.rows.E; t.next()) {
        const Tile tile(a, s, t);
        const bool sums = tile.rows > 0;
        if (!me.takes(sums) || (!sums && ADD)) continue;
        if (!sums) {
            const int r0 = tile.m0 + rank * 128;
            put_zeros(static_cast<uint16_t*>(a.g.out) + (int64_t(tile.e) * a.g.m + r0) * a.g.n + tile.n0, a.g.n,
                      min(128, a.g.m - r0), min(tile.blocks * 128, a.g.n - tile.n0), warp % 4, me.lane);
            __syncwarp();
            continue;
        }
        const int m0 = tile.m0 + me.first;
        const int width = m0 < a.g.m ? min(tile.blocks * 128, a.g.n - tile.n0) : 0;  // columns of the warp's rows
        // accumulate: the lane's row, on its way to L2 beside the products
        const uint16_t* old =
            static_cast<const uint16_t*>(a.g.out) + (int64_t(tile.e) * a.g.m + m0 + me.lane) * a.g.n + tile.n0;
        const bool add = ADD && m0 + me.lane < a.g.m;
        if (add)
            for (int c = 0; c < width; c += kCols) asm volatile("prefetch.global.L2 [%0];" ::"l"(old + c));
        if (!me.wait(a.g.rows.status)) break;
        if (width == 0) me.release();
        for (int c0 = 0; c0 < width; c0 += kPieces * kCols) {
            uint32_t w[kPieces][32];
#pragma unroll
            for (int i = 0; i < kPieces; i++) {
                const int c = c0 + i * kCols;
                if (c >= width) break;
                uint32_t r[64];
                tmem_load32(me.columns(c), r);
                tmem_load32(me.columns(c + 32), r + 32);
                tmem_wait(r, 64);
                if constexpr (ADD) {
                    // by all lanes, zeros in those past the matrix, and together again behind: the next piece is loaded from
                    // the accumulator by the whole warp, which must not have parted at a last row tile's end
                    uint4 x[8];
#pragma unroll
                    for (int j = 0; j < 8; j++)
                        x[j] = add && c + j * 8 < width ? *reinterpret_cast<const uint4*>(old + c + j * 8)
                                                        : make_uint4(0, 0, 0, 0);
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        float f[8];
                        unpack8(x[j], f);
#pragma unroll
                        for (int l = 0; l < 8; l++)
                            r[j * 8 + l] = __float_as_uint(__uint_as_float(r[j * 8 + l]) + f[l]);
                    }
                }
#pragma unroll
                for (int j = 0; j < 32; j++) w[i][j] = pack_sums(r + 2 * j);
            }
            if (c0 + kPieces * kCols >= width) me.release();
#pragma unroll
            for (int i = 0; i < kPieces; i++) {
                const int c = c0 + i * kCols;
                if (c >= width) break;
                if (me.lane == 0) bulk_wait_read<0>();  // the store before has read the buffer
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; j++)
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(mine + ((j ^ (me.lane & 7)) << 4)),
                                 "r"(w[i][4 * j]), "r"(w[i][4 * j + 1]), "r"(w[i][4 * j + 2]), "r"(w[i][4 * j + 3])
                                 : "memory");
                fence_proxy_async();
                __syncwarp();
                if (me.lane == 0) {
                    tma_store_3d(map_out, tile.n0 + c, m0, tile.e, buffer);
                    bulk_commit();
                }
                __syncwarp();
            }
        }
    }
    if (me.lane == 0) bulk_wait_all();
}

template <typename T, bool ADD>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    weight_grad_kernel(const __grid_constant__ GradArgs a, const __grid_constant__ GradMaps maps,
                       const __grid_constant__ CUtensorMap map_out) {
    extern __shared__ uint8_t raw[];
    uint8_t* base = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);  // slots on swizzle atoms
    const uint32_t slots = smem_addr(base);
    PairShared* s = reinterpret_cast<PairShared*>(base + a.slots * kSlot + (kFp32<T> ? 0 : kStaging));
    const int warp = threadIdx.x / 32, rank = int(cluster_rank());
    pair_start(s, a.g.rows, 0, 0, kPairEpilogueWarps / 2);
    if (warp == 0) {
        load_role<T, false>(a, s, slots, rank, maps.a);
    } else if (warp == 2) {
        load_role<T, true>(a, s, slots, rank, maps.b);
    } else if (warp == 1) {
        if (rank == 0) mma_role<T>(a, s, slots);
    } else if (warp >= 4) {
        if constexpr (kFp32<T>)
            epilogue_fp32<ADD>(a, s, rank, warp);
        else
            epilogue_bf16<ADD>(a, s, slots + a.slots * kSlot, rank, warp, &map_out);
    }
    pair_end(s);
}

}  // namespace

cudaError_t launch_weight_grad(const LaunchCtx& ctx, const WeightGrad& grad) {
    auto kern = grad.fp32 ? (grad.accumulate ? weight_grad_kernel<float, true> : weight_grad_kernel<float, false>)
                          : (grad.accumulate ? weight_grad_kernel<uint16_t, true> : weight_grad_kernel<uint16_t, false>);
    // first: it makes the device's context current in a thread that has made no CUDA call yet, and the maps need one
    const cudaError_t err = allow_shared_memory(kern, kPairShared);
    if (err != cudaSuccess) return err;
    WeightGrad g = grad;
    if (g.fp32) g.a = grad.b, g.m = grad.n, g.b = grad.a, g.n = grad.m;
    GradMaps maps{};
    CUtensorMap map_out{};
    const uint64_t rows = uint64_t(g.rows.rows), da[2] = {uint64_t(g.m), rows}, db[2] = {uint64_t(g.n), rows};
    const uint64_t dout[3] = {uint64_t(g.n), uint64_t(g.m), uint64_t(g.rows.E)};
    const uint32_t bout[3] = {64, 32, 1};
    for (int i = 0; i < kBoxes && rows > 0; i++) {  // without rows nothing is loaded
        const uint32_t box[2] = {64, uint32_t(kPairK) >> i};
        if (!make_map_bf16(&maps.a[i], g.a, 2, da, box) || !make_map_bf16(&maps.b[i], g.b, 2, db, box))
            return cudaErrorInvalidValue;
    }
    if (!g.fp32 && !make_map_bf16(&map_out, g.out, 3, dout, bout)) return cudaErrorInvalidValue;
    // as many slots as fit: a sixth makes 128 ragged experts in bf16 563 -> 533 us, a seventh in fp32 nothing
    const int E = g.rows.E, slots = g.fp32 || shared_bytes<uint16_t>(6, E) <= kPairShared ? 6 : 5;
    const size_t smem = g.fp32 ? shared_bytes<float>(slots, E) : shared_bytes<uint16_t>(slots, E);
    const GradArgs a{g, (g.m + kTile - 1) / kTile, (g.n + kTile - 1) / kTile, slots};
    return launch_pairs(ctx, kern, smem, a, maps, map_out);
}

}  // namespace moe
