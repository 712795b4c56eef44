// expert_gemm_bf16.cu -- the products of a dispatched layout's bf16 rows with their expert's weights.
//
//   plain     out[r, j] = sum_k a[r, k] w(e, j, k), weights [E, n, k] or [E, k, n]
//   SwiGLU    h = up * silu(gate) of two such products
//   dSwiGLU   the gradient of gate and up from such a product
//
// Persistent pairs of SMs, each walking over tiles of 256 columns x up to 288 rows of one expert. The weights are the M
// side of the products, 128 columns in each block (SwiGLU: 64 gate columns and the 64 up columns beside them), and the
// rows the N side, half of them in each block: N follows the expert's rows in steps of 32, so that few rows, or a few more
// than a tile, cost little more than they are. Warps have roles:
//   0      issues the loads of a ring of slots of 64 values of k, by tensor maps in the 128-byte swizzle (out-of-range
//          rows, columns and k read as zero); weights [E, k, n] are read as they lie and multiplied along their columns
//   1      of the leading block issues the products of both
//   4..11  take the accumulator (columns are its lanes) through shared memory to rows, and finish these
// Tiles run with the row tiles of one column block next to each other, so a weight tile comes from DRAM once. Two
// accumulators: the next tile's products run beside the epilogue. Every wait is bounded (MOE_ERR_TIMEOUT).
//
// What it measured (one GB300, single passes; 6777 GB/s is the copy bandwidth, cuBLAS reaches 1.92 PFLOP/s):
//   8 experts of 8192 rows, 4096 x 4096:    1165 us either way of the weights, 1.89 PFLOP/s
//   256 experts of 256 rows, 7168 -> 1024:  SwiGLU 1280 us, 6.7 TB/s: bound by reading the weights
//   the same with 256 +- 16 rows:           1330 us, 1370 with gate and up kept: half of the experts are in a tile of 288
//   128 experts of 512 +- 21 rows:          dSwiGLU 4096 -> 768 325 us, 1536 -> 4096 530 us, 1.55 PFLOP/s
//   128 experts of 32 rows, 4096 -> 2048:   333 us, 6.6 TB/s
//   8 experts of one row, SwiGLU 4096 -> 768: 18 us, of which 4.5 are the kernel's start
// A slot takes 345 ns with 256 rows (the products alone some 290) and 277 with 192, where what an SM takes in from L2 bounds
// it: 53 bytes a clock. The ring hides the rest of its latency: 6 slots of 256 rows for 5 make the ragged products 3 to 5 %
// faster. Under the power limit (1.38 kW) long runs are some 10 % slower.
#include <cstdint>
#include <type_traits>

#include "expert_pair.cuh"

namespace moe {
namespace {

// Rows of a tile beyond 256 are the N side of a second product on the same weights: of 288 rows, 160 and 128. The accumulators
// of a pair's tiles lie at the two ends of tensor memory in turn; where two of them meet, in 64 columns at most, the epilogue
// reads these first, and the next tile's products wait for that alone.
constexpr int kWideFirst = 160;
constexpr int kChunkRows = 16;  // rows of the accumulator that a group of epilogue warps takes at a time
static_assert(2 * kWideRows - int(kPairTmemColumns) <= 4 * kChunkRows, "two pieces of both groups are what may meet");
constexpr int kCols = 256;
constexpr uint32_t kStaged = kChunkRows * 128 * 4;           // ... of a block's 128 columns in fp32
constexpr uint32_t kStaging = 2 * kStaged;                   // two groups of four epilogue warps
// Bytes of the ring: what is left, in swizzle atoms.
constexpr uint32_t ring_bytes(int E) {
    return uint32_t(kPairShared - 1024 - kStaging - pair_shared_bytes(E)) / 1024 * 1024;
}
static_assert(ring_bytes(MOE_MAX_EXPERTS) >= 6 * 2 * kPairBytes, "six slots of tiles of 256 rows");
static_assert(ring_bytes(MOE_MAX_EXPERTS) >= 5 * (kPairBytes + kWideRows * 64), "five slots of the largest tiles");

struct GemmArgs {
    RowGemm g;
    int chunks;   // slots per tile: ceil(k / kPairK)
    int tiles_n;  // column tiles
    uint32_t ring;
};

struct Tile {
    int e, n0, row0, rows;  // expert, first column, first row, rows
    // N of the products; each block loads half of it
    __device__ __forceinline__ int n() const { return (rows + 31) & ~31; }
    __device__ __forceinline__ bool wide() const { return n() > 256; }
    __device__ __forceinline__ int first() const { return wide() ? kWideFirst : n(); }  // N of the first product
    // The first column of the accumulator of the i-th of a pair's tiles.
    __device__ __forceinline__ int column(int i) const { return i & 1 ? int(kPairTmemColumns) - max(n(), 256) : 0; }
};

template <RowOp OP>
constexpr int kTileCols = OP == RowOp::kSwiglu ? kCols / 2 : kCols;  // columns of the result in a tile

template <RowOp OP>
__device__ __forceinline__ Tile find_tile(const GemmArgs& a, PairShared* s, int t) {
    const int E = a.g.rows.E;
    const int* prefix = s->prefix();
    int lo = 0, hi = E;  // prefix[lo] * tiles_n <= t < prefix[hi] * tiles_n
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (int64_t(prefix[mid]) * a.tiles_n <= t)
            lo = mid;
        else
            hi = mid;
    }
    const int rows_t = prefix[lo + 1] - prefix[lo];
    const int i = int(t - int64_t(prefix[lo]) * a.tiles_n);
    int col = i, m = 0;
    if (rows_t > 1) {
        // the row tiles of a column turn from one round of the pairs to the next: the last of an expert is smaller, and the
        // same pairs would get it each time and run ahead of those that read the same weights (480 rows: 604 us, not 700)
        col = i / rows_t, m = i - col * rows_t;
        m = (m + (t - m) / int(gridDim.x / 2)) % rows_t;
    }
    // an expert's rows are shared out evenly among its tiles, in steps of 32
    const int count = s->count(E)[lo], each = (count + rows_t - 1) / rows_t;
    const int step = (each + 31) & ~31;
    const int first = min(m * step, count);
    return Tile{uniform(lo), uniform(col * kTileCols<OP>), uniform(s->base(E)[lo] + first),
                uniform(min(step, count - first))};
}

// Bytes of a slot, a multiple of the swizzle's atoms, and how many there are: by the largest tile. One token's 8 experts of
// 2 x 768 x 4096: 18.4 us, with slots of 32 KB 20.0; 128 experts of 32 rows, 4096 x 2048: 331 and 349 us.
__device__ __forceinline__ uint32_t slot_bytes(const PairShared* s) { return kPairBytes + uint32_t((s->most + 31) & ~31) * 64; }
__device__ __forceinline__ int ring_slots(const GemmArgs& a, uint32_t slot) { return min(kPairSlots, int(a.ring / slot)); }

constexpr int kBoxes = 4;
struct RowMaps {
    CUtensorMap a[kBoxes];  // boxes of 64 values x 128, 64, 32, 16 rows
};

// A whole warp; one lane issues, with operands that are the same in all lanes.
template <RowOp OP, bool KN>
__device__ __forceinline__ void load_role(const GemmArgs& a, PairShared* s, uint32_t slots, int rank, const RowMaps& maps,
                                          const CUtensorMap* map_w) {
    const int pairs = gridDim.x / 2, tiles = s->tiles * a.tiles_n;
    const uint32_t own = smem_addr(s->full), counted = leaders(own), empty = smem_addr(s->empty);
    const uint32_t leader = elect_one();
    const uint32_t slot_size = uniform(slot_bytes(s));
    const int stages = uniform(ring_slots(a, slot_size));
    int st = 0;
    uint32_t ph = 0;
    for (int t = blockIdx.x / 2; t < tiles; t += pairs) {
        const Tile tile = find_tile<OP>(a, s, t);
        const int half = tile.n() / 2, first = tile.first() / 2;  // of the block; those of the first product
        const int n0 = tile.n0 + rank * (kTileCols<OP> / 2);
        const uint32_t bytes = 2 * (kPairBytes + half * 128);
        for (int c = 0; c < a.chunks; c++) {
            if (!pair_wait_warp(s, a.g.rows.status, empty + 8 * st, ph ^ 1)) return;
            if (leader) {
                const uint32_t bar = counted + 8 * st, slot = slots + st * slot_size;
                const int k0 = c * kPairK;
                if (rank == 0) mbar_expect_tx(own + 8 * st, bytes);
                if constexpr (KN) {
                    pair_load_3d(slot, map_w, n0, k0, tile.e, bar);
                    pair_load_3d(slot + kPairBytes / 2, map_w, n0 + 64, k0, tile.e, bar);
                } else {
                    // (k, column, half, expert); SwiGLU: 64 columns of both halves
                    pair_load_4d(slot, map_w, k0, n0, 0, tile.e, bar);
                }
                uint32_t to = slot + kPairBytes;
                const auto load_rows = [&](int row, int count) {
#pragma unroll
                    for (int i = 0; i < kBoxes; i++) {
                        const int box = 128 >> i;
                        if (count & box) {
                            pair_load_2d(to, &maps.a[i], k0, row, bar);
                            to += box * 128, row += box;
                        }
                    }
                };
                load_rows(tile.row0 + rank * first, first);
                if (half > first) load_rows(tile.row0 + 2 * first + rank * (half - first), half - first);
            }
            __syncwarp();
            if (++st == stages) st = 0, ph ^= 1;
        }
    }
    pair_drain(s, a.g.rows.status, st, ph, stages);
}

// A whole warp of the leading block; one lane issues.
template <RowOp OP, bool KN>
__device__ __forceinline__ void mma_role(const GemmArgs& a, PairShared* s, uint32_t slots) {
    const uint64_t da = KN ? desc_mn128(slots) : desc_k128(slots), db = desc_k128(slots + kPairBytes);
    const uint32_t full = smem_addr(s->full), empty = smem_addr(s->empty), tmem = uniform(s->tmem);
    const int pairs = gridDim.x / 2, tiles = s->tiles * a.tiles_n;
    const int last = (a.g.k - (a.chunks - 1) * kPairK + 15) / 16;  // steps of 16 in the last slot
    const uint32_t leader = elect_one();
    const uint32_t slot_size = uniform(slot_bytes(s));
    const int stages = uniform(ring_slots(a, slot_size));
    int st = 0, n_tile = 0, edge = 0;
    uint32_t ph = 0;
    for (int t = blockIdx.x / 2; t < tiles; t += pairs, n_tile++) {
        const Tile tile = find_tile<OP>(a, s, t);
        const uint32_t idesc = pair_idesc_bf16(tile.first(), KN, false);
        const uint32_t idesc2 = pair_idesc_bf16(kWideRows - kWideFirst, KN, false);
        const int acc = n_tile & 1, column = tile.column(n_tile);
        const uint32_t d = tmem + column;
        if (!pair_wait_cluster(s, a.g.rows.status, smem_addr(&s->acc_empty[acc]), (n_tile >> 1 & 1) ^ 1)) return;
        // the tile before, at the other end
        if (n_tile > 0 && (acc == 0 ? tile.n() > edge : column < edge) &&
            !pair_wait_cluster(s, a.g.rows.status, smem_addr(&s->top_empty[acc ^ 1]), (n_tile - 1) >> 1 & 1))
            return;
        edge = acc == 0 ? tile.n() : column;  // where this one ends, towards the middle
        tc_fence_after();
        // a loop for either kind of tile: a branch in a slot's products costs every slot some 10 ns
        const auto products = [&](auto wide) {
            for (int c = 0; c < a.chunks; c++) {
                if (!pair_wait_warp(s, a.g.rows.status, full + 8 * st, ph)) return false;
                tc_fence_after();
                const uint32_t off = st * (slot_size / 16);
                const int steps = c + 1 < a.chunks ? 4 : last;
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    if (j >= steps) break;
                    // 16 values of k: 32 bytes further in the rows; or 16 rows of 128 bytes
                    const uint64_t w = da + off + (KN ? 128 : 2) * j, r = db + off + 2 * j;
                    pair_mma_bf16(leader, d, w, r, idesc, c > 0 || j > 0);
                    if constexpr (wide.value)
                        pair_mma_bf16(leader, d + kWideFirst, w, r + kWideFirst / 2 * 8, idesc2, c > 0 || j > 0);
                }
                pair_commit(leader, empty + 8 * st);
                if (c + 1 == a.chunks) pair_commit(leader, smem_addr(&s->acc_full[acc]));
                if (++st == stages) st = 0, ph ^= 1;
            }
            return true;
        };
        if (!(tile.wide() ? products(std::true_type()) : products(std::false_type()))) return;
    }
}

__device__ __forceinline__ uint2 pack4(float4 v) { return make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w)); }
__device__ __forceinline__ uint2 ld_v2(const void* p) {  // of what may be written in place
    uint2 v;
    asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

template <RowOp OP>
__device__ __forceinline__ void epilogue_role(const GemmArgs& a, PairShared* s, float* staging, int rank, int warp) {
    const int lane = threadIdx.x % 32, quad = warp % 4, group = (warp - 4) / 4;
    const uint32_t tmem = s->tmem + (uint32_t(quad * 32) << 16);  // the 32 lanes that the warp may read
    const int pairs = gridDim.x / 2, tiles = s->tiles * a.tiles_n, n = a.g.n;
    float* stage = staging + group * (kStaged / 4);
    constexpr int kPieces = 2;  // taken before they are written
    const bool meet = s->most > 256;
    int n_tile = 0;
    for (int t = blockIdx.x / 2; t < tiles; t += pairs, n_tile++) {
        const Tile tile = find_tile<OP>(a, s, t);
        const int acc = n_tile & 1, times = tile.n() / (2 * kChunkRows), column = tile.column(n_tile);
        const int n0 = tile.n0 + rank * (kTileCols<OP> / 2);
        if (!group_all(group, pair_wait(s, a.g.rows.status, smem_addr(&s->acc_full[acc]), n_tile >> 1 & 1))) return;
        tc_fence_after();
        const uint32_t done = leaders(smem_addr(&s->acc_empty[acc])), top = leaders(smem_addr(&s->top_empty[acc]));
        if (n0 >= n) {  // nothing to finish
            if (lane == 0) {
                if (meet) mbar_arrive_cluster(top);
                mbar_arrive_cluster(done);
            }
            continue;
        }
        // from the end that the next tile's accumulator may meet
        for (int i0 = 0; i0 < times; i0 += kPieces) {
            int j0[kPieces];
            uint2 gate[kPieces][4], up[kPieces][4];
            float v[kPieces][kChunkRows];
#pragma unroll
            for (int x = 0; x < kPieces; x++) {
                const int i = i0 + x;
                j0[x] = i < times ? ((acc ? i : times - 1 - i) * 2 + group) * kChunkRows : tile.rows;
                if constexpr (OP == RowOp::kDswiglu) {
                    // gate and up of the rows and columns that this lane will finish, on their way beside the accumulator
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const int j = j0[x] + quad * 4 + i, col = n0 + lane * 4;
                        if (j >= tile.rows || col >= n) continue;
                        const uint16_t* p = a.g.gate_up + (int64_t(tile.row0) + j) * 2 * n + col;
                        gate[x][i] = ld_v2(p);
                        up[x][i] = ld_v2(p + n);
                    }
                }
            }
            __syncwarp();
#pragma unroll
            for (int x = 0; x < kPieces; x++)
                if (j0[x] < tile.rows) tmem_load16(tmem + column + j0[x], v[x]);
            const bool met = meet && i0 == 0, last = i0 + kPieces >= times;
            if (met || last) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (met) mbar_arrive_cluster(top);
                    if (last) mbar_arrive_cluster(done);
                }
            }
#pragma unroll
            for (int x = 0; x < kPieces; x++) {
                if (j0[x] >= tile.rows) continue;
                group_sync(group);  // what was there before has been read
#pragma unroll
                for (int j = 0; j < kChunkRows; j++) stage[j * 128 + quad * 32 + lane] = v[x][j];
                group_sync(group);
                if constexpr (OP == RowOp::kSwiglu) {
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const int j = quad * 4 + i * 2 + lane / 16, c = lane % 16 * 4, col = n0 + c;
                        if (j0[x] + j >= tile.rows || col >= n) continue;
                        const int64_t r = int64_t(tile.row0) + j0[x] + j;
                        const float4 g = *reinterpret_cast<const float4*>(stage + j * 128 + c);
                        const float4 u = *reinterpret_cast<const float4*>(stage + j * 128 + 64 + c);
                        st_v2(a.g.out + r * n + col, pack4(make_float4(swiglu(g.x, u.x), swiglu(g.y, u.y), swiglu(g.z, u.z),
                                                                       swiglu(g.w, u.w))));
                        if (a.g.gate_up) {
                            st_v2(a.g.gate_up + r * 2 * n + col, pack4(g));
                            st_v2(a.g.gate_up + (r * 2 + 1) * n + col, pack4(u));
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const int j = quad * 4 + i, col = n0 + lane * 4;
                        if (j0[x] + j >= tile.rows || col >= n) continue;
                        const int64_t r = int64_t(tile.row0) + j0[x] + j;
                        const float4 sums = *reinterpret_cast<const float4*>(stage + j * 128 + lane * 4);
                        if constexpr (OP == RowOp::kPlain) {
                            st_v2(a.g.out + r * n + col, pack4(sums));
                        } else {
                            // Rounded to bf16, from fp32 sums and factors: the two products that read these gradients
                            // next (of the rows, transposed, and of the gate and up weights) take bf16. What goes
                            // through both roundings is 0.0023 off in norm, 0.0017 with these values kept in fp32; that
                            // would be twice the bytes written here and read twice.
                            float4 dg, du;
                            dswiglu(bf16_lo(gate[x][i].x), bf16_lo(up[x][i].x), sums.x, &dg.x, &du.x);
                            dswiglu(bf16_hi(gate[x][i].x), bf16_hi(up[x][i].x), sums.y, &dg.y, &du.y);
                            dswiglu(bf16_lo(gate[x][i].y), bf16_lo(up[x][i].y), sums.z, &dg.z, &du.z);
                            dswiglu(bf16_hi(gate[x][i].y), bf16_hi(up[x][i].y), sums.w, &dg.w, &du.w);
                            st_v2(a.g.out + r * 2 * n + col, pack4(dg));
                            st_v2(a.g.out + (r * 2 + 1) * n + col, pack4(du));
                        }
                    }
                }
            }
        }
    }
}

template <RowOp OP, bool KN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    row_gemm_kernel(const __grid_constant__ GemmArgs a, const __grid_constant__ RowMaps maps,
                    const __grid_constant__ CUtensorMap map_w) {
    extern __shared__ uint8_t raw[];
    uint8_t* base = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);  // slots on swizzle atoms
    const uint32_t slots = smem_addr(base);
    float* staging = reinterpret_cast<float*>(base + a.ring);
    PairShared* s = reinterpret_cast<PairShared*>(base + a.ring + kStaging);
    const int warp = threadIdx.x / 32, rank = int(cluster_rank());
    pair_start(s, a.g.rows, a.tiles_n, a.chunks, kPairEpilogueWarps);
    if (warp == 0) {
        load_role<OP, KN>(a, s, slots, rank, maps, &map_w);
    } else if (warp == 1) {
        if (rank == 0) mma_role<OP, KN>(a, s, slots);
    } else if (warp >= 4) {
        epilogue_role<OP>(a, s, staging, rank, warp);
    }
    pair_end(s);
}

template <RowOp OP, bool KN>
cudaError_t launch(const LaunchCtx& ctx, const RowGemm& g) {
    auto kern = row_gemm_kernel<OP, KN>;
    // first: it makes the device's context current in a thread that has made no CUDA call yet, and the maps need one
    const cudaError_t err = allow_shared_memory(kern, kPairShared);
    if (err != cudaSuccess) return err;
    constexpr uint64_t halves = OP == RowOp::kSwiglu ? 2 : 1;
    const uint64_t k = uint64_t(g.k), n = uint64_t(g.n), E = uint64_t(g.rows.E);
    const uint64_t da[2] = {k, uint64_t(g.rows.rows)}, dnk[4] = {k, n, halves, E}, dkn[3] = {n, k, E};
    const uint32_t bnk[4] = {kPairK, uint32_t(128 / halves), halves, 1}, bkn[3] = {64, kPairK, 1};
    RowMaps maps;
    CUtensorMap map_w;
    for (int i = 0; i < kBoxes; i++) {
        const uint32_t box[2] = {kPairK, 128u >> i};
        if (!make_map_bf16(&maps.a[i], g.a, 2, da, box)) return cudaErrorInvalidValue;
    }
    if (!(KN ? make_map_bf16(&map_w, g.w, 3, dkn, bkn) : make_map_bf16(&map_w, g.w, 4, dnk, bnk)))
        return cudaErrorInvalidValue;
    const GemmArgs a{g, (g.k + kPairK - 1) / kPairK, (g.n + kTileCols<OP> - 1) / kTileCols<OP>, ring_bytes(g.rows.E)};
    return launch_pairs(ctx, kern, 1024 + a.ring + kStaging + pair_shared_bytes(g.rows.E), a, maps, map_w);
}

}  // namespace

cudaError_t launch_row_gemm(const LaunchCtx& ctx, const RowGemm& g) {
    if (g.op == RowOp::kSwiglu) return launch<RowOp::kSwiglu, false>(ctx, g);
    if (g.op == RowOp::kDswiglu) return launch<RowOp::kDswiglu, true>(ctx, g);
    return g.kn ? launch<RowOp::kPlain, true>(ctx, g) : launch<RowOp::kPlain, false>(ctx, g);
}

}  // namespace moe
