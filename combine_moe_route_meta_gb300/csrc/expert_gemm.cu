// expert_gemm.cu -- the product of a dispatched layout's NVFP4 rows with their expert's weights.
//
//   out[r, n] = bf16(alpha[e] * sum_k a[r, k] w[e, n, k])
//   SwiGLU:  h = silu(gate) * up of two such products, quantised to NVFP4
//
// Persistent CTAs, one per SM, each walking over tiles of 128 rows x 256 columns (SwiGLU: 128 gate columns
// and the 128 up columns beside them) of one expert. Warps have roles:
//   0      issues the loads of a ring of kStages slots, each 256 values of K: codes by tensor maps in the
//          128-byte swizzle (out-of-range rows and columns read as zero), weight scales (whole 512-byte
//          tiles) by bulk copies, and the rows' scales too where their 128-row tiles are the layout's own
//   1      copies a slot's scale tiles to tensor memory and issues its block-scaled products
//   2, 3   gather the rows' scales into the tile layout where rows start inside a tile or scales are row-major
//   4..11  turn the fp32 accumulator into the output; they free it as soon as they hold its last columns
// Tiles run with the row tiles of one column block next to each other, so a weight tile comes from DRAM once
// and from L2 for the others. Every wait is bounded (MOE_ERR_TIMEOUT).
//
// Why so, and what it measured (one GB300; 6782 GB/s is the copy bandwidth):
//   256 experts, k 7168 -> 1024 -> 7168 (SwiGLU and the product after it), weights of 3.1 GB
//     128 tokens top-8, masked:   461 us, 6.8 TB/s: bound by reading the weights once
//     8192 tokens top-8:          840 to 880 us, 5.1 TB/s and 2.9 TFLOP at 3.4 PFLOP/s, at the power limit
//   128 experts, k 768 -> 4096, 2048 tokens top-8 skewed: 67 us, 5.5 TB/s
//   16 experts, k 4096 -> 704 -> 4096, 1501 tokens top-4: 46 us
// With many rows an expert the first product's bound is what an SM takes in from L2: a tile brings 128 + 256 rows of
// codes for 128 x 256 results, 56 bytes a clock and SM between two tile ends, 15.0 TB/s over a whole launch, while the
// tensor core is busy for 55 % and DRAM for 61 % of the time. Three ways to take in less were not built: wider tiles (the
// scales of the four slots fill the half of tensor memory beside the accumulator, but two sets in turn would leave 384
// columns for it), two products of 128 rows on one slot's weights, and pairs of SMs that share a weight tile (which round
// an expert's rows up to 256). The second product, with its larger output, is bound by DRAM. One lane elected from a converged warp issues the products:
// issued by a divergent lane they cost 60 ns each, and the first case above took 608 us.
#include <cstdint>

#include "expert_rows.cuh"
#include "experts_launch.h"
#include "tcgen05.cuh"
#include "tensor_map.h"

namespace moe {
namespace {

constexpr int kTileM = 128;
constexpr int kTileN = 256;
constexpr int kChunk = 256;                           // values of K per slot: 128 bytes of codes a row
constexpr int kStages = 4;
constexpr int kWarps = 12;
constexpr int kThreads = kWarps * 32;
constexpr int kLoaderWarps = 2;                       // of row scales, taking slots in turn
static_assert(kStages % kLoaderWarps == 0, "a loader's next slot is less than a round of the ring ahead");
constexpr int kEpilogueWarps = 8;
constexpr uint32_t kBytesA = kTileM * 128;            // codes of a slot
constexpr uint32_t kBytesB = kTileN * 128;
constexpr uint32_t kBytesSfA = kTileM * (kChunk / 16);  // scales of a slot
constexpr uint32_t kBytesSfB = kTileN * (kChunk / 16);
constexpr uint32_t kSlot = kBytesA + kBytesB + kBytesSfA + kBytesSfB;
constexpr uint32_t kTmemColumns = 512;
constexpr uint32_t kTmemScales = kTileN;              // after the accumulator: 16 + 32 columns for every slot, so
constexpr uint32_t kTmemScaleSet = 64;                // that a slot's scales live as long as the slot itself
static_assert(kTmemScales + kStages * kTmemScaleSet <= kTmemColumns, "scales of every slot in tensor memory");

struct GemmArgs {
    ExpertGemm g;
    int chunks;       // slots per tile: ceil(k / kChunk)
    int tiles_n;
    bool sf_bulk_ok;  // the rows' scales are in 128 x 4 tiles at a 16-byte aligned address
    bool wide_out;    // out is 32-byte aligned
};

struct Tile {
    int e, n0, row0, rows;  // expert, first column (of gate), first row, rows
};

struct Shared {
    uint64_t full[kStages], empty[kStages], acc_full, acc_empty;
    uint32_t tmem;
    int dead;       // a wait gave up
    int tiles;
    // behind: prefix [E + 1], row tiles of the experts before e; base [E], first rows; last [E], rows of the last tile - 1
    __device__ __forceinline__ int* prefix() { return reinterpret_cast<int*>(this + 1); }
    __device__ __forceinline__ int* base(int E) { return prefix() + E + 1; }
    __device__ __forceinline__ uint8_t* last(int E) { return reinterpret_cast<uint8_t*>(base(E) + E); }
};
constexpr size_t shared_bytes(int E) { return sizeof(Shared) + size_t(E + 1) * 4 + size_t(E) * 5; }
static_assert(1024 + kStages * kSlot + shared_bytes(MOE_MAX_EXPERTS) <= 227 * 1024, "shared memory of an SM");

template <bool SWIGLU>
__device__ __forceinline__ Tile find_tile(const GemmArgs& a, Shared* s, int t) {
    const int* prefix = s->prefix();
    int lo = 0, hi = a.g.E;  // prefix[lo] * tiles_n <= t < prefix[hi] * tiles_n
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (int64_t(prefix[mid]) * a.tiles_n <= t)
            lo = mid;
        else
            hi = mid;
    }
    const int rows_t = prefix[lo + 1] - prefix[lo];
    const int i = int(t - int64_t(prefix[lo]) * a.tiles_n);
    const int m = i % rows_t;
    return Tile{lo, i / rows_t * (SWIGLU ? kTileN / 2 : kTileN), s->base(a.g.E)[lo] + m * kTileM,
                m + 1 < rows_t ? kTileM : s->last(a.g.E)[lo] + 1};
}

// Bounded wait; false (and the CTA marked dead) when it gave up or another role already had.
__device__ __forceinline__ bool wait_or_die(const GemmArgs& a, Shared* s, uint32_t bar, uint32_t parity) {
    if (mbar_wait(bar, parity)) return true;
    *const_cast<volatile int*>(&s->dead) = 1;
    set_status(a.g.status, MOE_ERR_TIMEOUT);
    return false;
}

// The same for a whole warp: every lane gets the same answer.
__device__ __forceinline__ bool warp_wait_or_die(const GemmArgs& a, Shared* s, uint32_t bar, uint32_t parity) {
    return __all_sync(kFullMask, wait_or_die(a, s, bar, parity));
}

template <bool SWIGLU>
__device__ __forceinline__ void load_role(const GemmArgs& a, Shared* s, uint32_t slots, bool sf_bulk,
                                          const CUtensorMap* map_a, const CUtensorMap* map_a32,
                                          const CUtensorMap* map_w) {
    const int k64 = a.g.k / 64;
    const int np128 = (a.g.n + 127) / 128;  // 128-row blocks of a weight matrix
    int st = 0;
    uint32_t ph = 0;
    for (int t = blockIdx.x; t < s->tiles; t += gridDim.x) {
        const Tile tile = find_tile<SWIGLU>(a, s, t);
        for (int c = 0; c < a.chunks; c++) {
            if (!wait_or_die(a, s, smem_addr(&s->empty[st]), ph ^ 1)) return;
            const uint32_t bar = smem_addr(&s->full[st]), slot = slots + st * kSlot;
            const uint32_t sfa = slot + kBytesA + kBytesB, sfb = sfa + kBytesSfA;
            const int q = min(4, k64 - 4 * c);  // 64-value steps of this slot
            const int nb = tile.n0 / 128;
            const bool second = SWIGLU || nb + 1 < np128;
            // Of a tile with up to 32 rows only 32 are read: in a masked layout what follows an expert's rows costs
            // DRAM bandwidth (256 experts, 4 rows each: 475 us with 128 rows, 461 us with 32). Boxes for 64 and 96 rows
            // gained nothing (prefill 861 -> 873 us). The slot's other rows keep what they hold: their results
            // are not looked at.
            const bool few = tile.rows <= kTileM / 4;
            mbar_expect_tx(bar, (few ? kBytesA / 4 : kBytesA) + kBytesB +
                                    q * 512 * ((sf_bulk ? 1 : 0) + (second ? 2 : 1)));
            tma_load_2d(slot, few ? map_a32 : map_a, c * 128, tile.row0, bar);
            // SwiGLU: dimensions (k, column, half, expert), 128 columns of both halves; else (k, column, 1, expert)
            tma_load_4d(slot + kBytesA, map_w, c * 128, tile.n0, 0, tile.e, bar);
            if (sf_bulk)
                bulk_load_announced(sfa, a.g.a_sf + (int64_t(tile.row0 / 128) * k64 + 4 * c) * 512, q * 512, bar);
            const int64_t block = SWIGLU ? int64_t(tile.e) * 2 * np128 + nb : int64_t(tile.e) * np128 + nb;
            bulk_load_announced(sfb, a.g.w_sf + (block * k64 + 4 * c) * 512, q * 512, bar);
            if (second)
                bulk_load_announced(sfb + kBytesSfB / 2,
                                    a.g.w_sf + ((block + (SWIGLU ? np128 : 1)) * k64 + 4 * c) * 512, q * 512, bar);
            if (++st == kStages) st = 0, ph ^= 1;
        }
    }
}

// What the products read in the first slot; a slot further, kSlot / 16 more.
struct Operands {
    uint64_t a, b, sfa, sfb0, sfb1;
};

// The products of a slot: q steps of 64 values, their scales first.
__device__ __forceinline__ void multiply_slot(const Operands& o, uint32_t off, uint32_t d, uint32_t ts, uint32_t idesc, int q,
                                              bool add) {
#pragma unroll
    for (int j = 0; j < 4; j++) {
        if (j >= q) break;
        tc_copy_scales(ts + j * 4, o.sfa + off + j * 32);
        tc_copy_scales(ts + 16 + j * 8, o.sfb0 + off + j * 32);
        tc_copy_scales(ts + 16 + j * 8 + 4, o.sfb1 + off + j * 32);
    }
#pragma unroll
    for (int j = 0; j < 4; j++) {
        if (j >= q) break;
        // 64 codes: 32 bytes further in the rows, 2 in the descriptor's units
        tc_mma_nvfp4(d, o.a + off + 2 * j, o.b + off + 2 * j, idesc, ts + j * 4, ts + 16 + j * 8, add || j > 0);
    }
}

// A whole warp; one lane issues.
template <bool SWIGLU>
__device__ __forceinline__ void mma_role(const GemmArgs& a, Shared* s, uint32_t slots) {
    const uint32_t tmem = s->tmem, sf = slots + kBytesA + kBytesB;
    const Operands o{desc_k128(slots), desc_k128(slots + kBytesA), desc_scales(sf), desc_scales(sf + kBytesSfA),
                     desc_scales(sf + kBytesSfA + kBytesSfB / 2)};
    const uint32_t full = smem_addr(s->full), empty = smem_addr(s->empty);
    const int q_last = a.g.k / 64 - 4 * (a.chunks - 1);
    const bool leader = elect_one();
    int st = 0, n_tile = 0;
    uint32_t ph = 0;
    for (int t = blockIdx.x; t < s->tiles; t += gridDim.x, n_tile++) {
        const Tile tile = find_tile<SWIGLU>(a, s, t);
        const uint32_t idesc = idesc_nvfp4(SWIGLU ? kTileN : min(kTileN, a.g.n - tile.n0));
        if (!warp_wait_or_die(a, s, smem_addr(&s->acc_empty), (n_tile & 1) ^ 1)) return;
        tc_fence_after();
        for (int c = 0; c < a.chunks; c++) {
            if (!warp_wait_or_die(a, s, full + 8 * st, ph)) return;
            tc_fence_after();
            if (leader) {
                const uint32_t off = st * (kSlot / 16), ts = tmem + kTmemScales + st * kTmemScaleSet;
                if (c + 1 < a.chunks || q_last == 4)
                    multiply_slot(o, off, tmem, ts, idesc, 4, c > 0);
                else
                    multiply_slot(o, off, tmem, ts, idesc, q_last, c > 0);
                tc_commit(empty + 8 * st);
                if (c + 1 == a.chunks) tc_commit(smem_addr(&s->acc_full));
            }
            __syncwarp();
            if (++st == kStages) st = 0, ph ^= 1;
        }
    }
    // the last slot's arrival is the last that is on its way to this CTA's memory
    if (n_tile > 0) warp_wait_or_die(a, s, empty + 8 * (st == 0 ? kStages - 1 : st - 1), st == 0 ? ph ^ 1 : ph);
}

// Row scales that are not whole tiles of the layout: a warp brings every second slot's, a lane those of four rows
// (16 bytes of a tile's line), with its next slot's (of the next tile too) on their way while it waits for one.
template <bool SWIGLU>
__device__ __forceinline__ void scale_role(const GemmArgs& a, Shared* s, uint32_t slots, int turn) {
    const int C = a.g.k / 16, k64 = a.g.k / 64, lane = threadIdx.x & 31;
    const bool tiles = a.g.scale_layout == MOE_SCALES_SWIZZLED_128X4;
    const int step = tiles ? 512 : 4;  // bytes from word to word
    const bool whole = !tiles && C % 16 == 0 && reinterpret_cast<uintptr_t>(a.g.a_sf) % 16 == 0;  // a slot's words at once
    int t = blockIdx.x, c = turn;  // of the words to load next
    int64_t src[4];
    bool fresh = true;
    uint32_t next[4][4];
    int st = turn;
    uint32_t ph = 0;
    for (bool first = true;; first = false) {
        uint32_t v[4][4];
        const bool have = !first && t < s->tiles;
        if (!first) {
#pragma unroll
            for (int j = 0; j < 4; j++)
#pragma unroll
                for (int w = 0; w < 4; w++) v[j][w] = next[j][w];
            if (!have) return;
            for (c += kLoaderWarps; c >= a.chunks; c -= a.chunks) t += gridDim.x, fresh = true;
        } else {
            for (; c >= a.chunks; c -= a.chunks) t += gridDim.x;
        }
        if (t < s->tiles) {
            if (fresh) {
                const Tile tile = find_tile<SWIGLU>(a, s, t);
#pragma unroll
                for (int j = 0; j < 4; j++)
                    src[j] = act_sf_index(a.g.scale_layout, min(int64_t(tile.row0) + lane + 32 * j, a.g.rows - 1), 0, C);
                fresh = false;
            }
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const uint8_t* from = a.g.a_sf + src[j] + int64_t(c) * 4 * step;
                if (whole) {
                    const uint4 u = __ldg(reinterpret_cast<const uint4*>(from));
                    next[j][0] = u.x, next[j][1] = u.y, next[j][2] = u.z, next[j][3] = u.w;
                } else {
#pragma unroll
                    for (int w = 0; w < 4; w++)
                        next[j][w] = c * 4 + w < k64 ? __ldg(reinterpret_cast<const uint32_t*>(from + w * step)) : 0u;
                }
            }
        }
        if (first) continue;
        if (!warp_wait_or_die(a, s, smem_addr(&s->empty[st]), ph ^ 1)) return;
        const uint32_t to = slots + st * kSlot + kBytesA + kBytesB + lane * 16;
#pragma unroll
        for (int w = 0; w < 4; w++)
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to + w * 512), "r"(v[0][w]), "r"(v[1][w]),
                         "r"(v[2][w]), "r"(v[3][w])
                         : "memory");
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&s->full[st]));
        st += kLoaderWarps;
        if (st >= kStages) st -= kStages, ph ^= 1;
    }
}

__device__ __forceinline__ void store_out16(uint16_t* dst, const uint32_t* v, float alpha, bool wide) {
    uint32_t w[8];
#pragma unroll
    for (int p = 0; p < 8; p++) w[p] = pack_bf16x2(alpha * __uint_as_float(v[2 * p]), alpha * __uint_as_float(v[2 * p + 1]));
    if (wide) {
        st_v8(dst, w);
    } else {
        st_v4(dst, make_uint4(w[0], w[1], w[2], w[3]));
        st_v4(dst + 8, make_uint4(w[4], w[5], w[6], w[7]));
    }
}

// One block of 16 SwiGLU outputs as codes and a scale byte.
__device__ __forceinline__ uint32_t quantise_h(const uint32_t* gate, const uint32_t* up, float alpha, float gs, uint2* codes) {
    float h[16];
#pragma unroll
    for (int j = 0; j < 16; j++) h[j] = swiglu(alpha * __uint_as_float(gate[j]), alpha * __uint_as_float(up[j]));
    uint32_t sf;
    *codes = quantise_block(h, gs, &sf);
    return sf;
}

template <bool SWIGLU>
__device__ __forceinline__ void epilogue_role(const GemmArgs& a, Shared* s, int warp) {
    const int lane = threadIdx.x & 31;
    const int quad = warp % 4, half = (warp - 4) / 4;  // a warp reads the 32 lanes of tensor memory that are its own
    const uint32_t tmem = s->tmem + (uint32_t(quad * 32) << 16);
    int n_tile = 0;
    for (int t = blockIdx.x; t < s->tiles; t += gridDim.x, n_tile++) {
        const Tile tile = find_tile<SWIGLU>(a, s, t);
        const float alpha = a.g.alpha ? __ldg(a.g.alpha + tile.e) : 1.0f;
        const int m = quad * 32 + lane;
        const bool valid = m < tile.rows;
        const int64_t r = int64_t(tile.row0) + m;
        if (!warp_wait_or_die(a, s, smem_addr(&s->acc_full), n_tile & 1)) return;
        tc_fence_after();
        // the warp's half of the tile to registers at once, so that the next tile's products can begin: 128
        // columns, with SwiGLU 64 gate columns and their up columns
        uint32_t r32[128];
#pragma unroll
        for (int c = 0; c < 4; c++)
            tmem_load32(tmem + (SWIGLU ? c / 2 * (kTileN / 2) + half * 64 + c % 2 * 32 : half * 128 + c * 32), r32 + c * 32);
        tmem_wait(r32, 128);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&s->acc_empty));
        if (!valid) continue;
        if constexpr (!SWIGLU) {
            const int col = tile.n0 + half * 128;
            uint16_t* dst = a.g.out + r * a.g.n + col;
#pragma unroll
            for (int c = 0; c < 8; c++)
                if (col + c * 16 < a.g.n) store_out16(dst + c * 16, r32 + c * 16, alpha, a.wide_out);
        } else {
            // 64 columns of h: 32 bytes of codes and one word of scales
            const int n = tile.n0 + half * 64;
            if (n >= a.g.n) continue;
            uint32_t sf = 0;
            uint2 q[4];
#pragma unroll
            for (int c = 0; c < 4; c++)
                sf |= quantise_h(r32 + c * 16, r32 + 64 + c * 16, alpha, a.g.h_scale, &q[c]) << (8 * c);
            uint8_t* dst = a.g.h + r * (a.g.n / 2) + n / 2;
            st_v4(dst, make_uint4(q[0].x, q[0].y, q[1].x, q[1].y));
            st_v4(dst + 16, make_uint4(q[2].x, q[2].y, q[3].x, q[3].y));
            *reinterpret_cast<uint32_t*>(a.g.h_sf + act_sf_index(a.g.scale_layout, r, n / 16, a.g.n / 16)) = sf;
        }
    }
}

template <bool SWIGLU>
__global__ void __launch_bounds__(kThreads, 1)
    expert_gemm_kernel(const __grid_constant__ GemmArgs a, const __grid_constant__ CUtensorMap map_a,
                       const __grid_constant__ CUtensorMap map_a32, const __grid_constant__ CUtensorMap map_w) {
    extern __shared__ uint8_t raw[];
    uint8_t* base = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);  // slots on swizzle atoms
    const uint32_t slots = smem_addr(base);
    Shared* s = reinterpret_cast<Shared*>(base + kStages * kSlot);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (warp == 1) tmem_alloc(smem_addr(&s->tmem), kTmemColumns);
    pdl_wait();

    // row tiles of every expert, their prefix sums, and whether all segments start on a tile of scales
    int ragged = 0;
    for (int e = threadIdx.x; e < a.g.E; e += kThreads) {
        const RowSpan r = expert_rows(a.g, e);
        s->prefix()[e + 1] = int((uint32_t(r.count) + kTileM - 1) / kTileM);
        s->base(a.g.E)[e] = int(r.base);
        s->last(a.g.E)[e] = uint8_t((uint32_t(r.count) + kTileM - 1) % kTileM);
        ragged |= r.count > 0 && r.base % 128 != 0;
    }
    const bool sf_bulk = !__syncthreads_or(ragged) && a.sf_bulk_ok;
    if (warp == 0) {
        int64_t sum = 0;
        for (int e0 = 0; e0 < a.g.E; e0 += 32) {
            int v = e0 + lane < a.g.E ? s->prefix()[e0 + lane + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(kFullMask, v, o);
                if (lane >= o) v += u;
            }
            if (e0 + lane < a.g.E) s->prefix()[e0 + lane + 1] = int(sum + v);
            sum += __shfl_sync(kFullMask, v, 31);
        }
        // Experts that share no row have at most so many row tiles, and their tiles of the output are counted in 31 bits
        // (checked on the host). Overlapping segments could have any number of both.
        if (sum > a.g.rows / kTileM + a.g.E) {
            if (lane == 0) set_status(a.g.status, MOE_ERR_INVALID_ARG);
            sum = 0;
        }
        if (lane == 0) {
            s->prefix()[0] = 0;
            s->tiles = int(sum) * a.tiles_n;
            s->dead = 0;
            for (int i = 0; i < kStages; i++) {
                mbar_init(smem_addr(&s->full[i]), sf_bulk ? 1 : 2);
                mbar_init(smem_addr(&s->empty[i]), 1);
            }
            mbar_init(smem_addr(&s->acc_full), 1);
            mbar_init(smem_addr(&s->acc_empty), kEpilogueWarps);
            mbar_fence_init();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    if (warp == 0) {
        if (lane == 0) load_role<SWIGLU>(a, s, slots, sf_bulk, &map_a, &map_a32, &map_w);
    } else if (warp == 1) {
        mma_role<SWIGLU>(a, s, slots);
    } else if (warp < 4) {
        if (!sf_bulk) scale_role<SWIGLU>(a, s, slots, warp - 2);
    } else {
        epilogue_role<SWIGLU>(a, s, warp);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*const_cast<volatile int*>(&s->dead) && threadIdx.x == 0) {
        // whatever is still in flight lands in this CTA's memory: give it time before that is freed
        const uint64_t t0 = global_ns();
        while (global_ns() - t0 < kDrainLimitNs) __nanosleep(1000);
    }
    __syncthreads();
    if (warp == 1) tmem_free(s->tmem, kTmemColumns);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
template <bool SWIGLU>
cudaError_t launch(const LaunchCtx& ctx, const ExpertGemm& g) {
    auto kern = expert_gemm_kernel<SWIGLU>;
    // first: it makes the device's context current in a thread that has made no CUDA call yet, and the maps need one
    const cudaError_t err = allow_shared_memory(kern, 1024 + size_t(kStages) * kSlot + shared_bytes(MOE_MAX_EXPERTS));
    if (err != cudaSuccess) return err;
    const uint64_t kb = uint64_t(g.k) / 2;
    CUtensorMap map_a, map_a32, map_w;
    const uint64_t da[2] = {kb, uint64_t(g.rows)}, dw[4] = {kb, uint64_t(g.n), SWIGLU ? 2u : 1u, uint64_t(g.E)};
    const uint32_t ba[2] = {128, kTileM}, ba32[2] = {128, kTileM / 4},
                   bw[4] = {128, SWIGLU ? kTileN / 2 : kTileN, SWIGLU ? 2u : 1u, 1};
    if (!make_map(&map_a, g.a, 2, da, ba) || !make_map(&map_a32, g.a, 2, da, ba32) || !make_map(&map_w, g.w, 4, dw, bw))
        return cudaErrorInvalidValue;
    const int cols = SWIGLU ? kTileN / 2 : kTileN;
    const GemmArgs a{g, (g.k + kChunk - 1) / kChunk, (g.n + cols - 1) / cols,
                     g.scale_layout == MOE_SCALES_SWIZZLED_128X4 && reinterpret_cast<uintptr_t>(g.a_sf) % 16 == 0,
                     reinterpret_cast<uintptr_t>(g.out) % 32 == 0};
    const size_t smem = 1024 + size_t(kStages) * kSlot + shared_bytes(g.E);
    return launch_pdl(ctx, kern, dim3(unsigned(ctx.num_sms)), dim3(kThreads), smem, a, map_a, map_a32, map_w);
}

}  // namespace

cudaError_t launch_expert_gemm(const LaunchCtx& ctx, const ExpertGemm& g) {
    return g.out == nullptr ? launch<true>(ctx, g) : launch<false>(ctx, g);
}

}  // namespace moe
