// moe_layer.cu -- a whole MoE layer for a few tokens in two kernels.
//
//   gate_up:  h(p) = silu(alpha1 W1g x) * (alpha1 W1u x) for every pair p = (token, slot), e its expert
//   down:     out[t] = bf16(sum over t's pairs of topk_weight * alpha2 * W2 h(p))
//
// Bound by reading each routed expert's weights once from DRAM, so the weights take the shortest way there is:
// tensor-map loads to shared memory, from which the tensor core reads them as they are. Weight rows are the
// M side of its products, the few tokens of an expert the N side.
//
// NVFP4 weights need NVFP4 on the other side too. A block of 16 values of x (or h) is a sum of five such blocks,
//   r_0 = x 2^s;  q_i = nvfp4(8^i r_i);  r_{i+1} = r_i - 8^-i q_i;   x 2^s ~ sum 8^-i q_i,
// each of which leaves at most 0.18 of the block's largest value (half of e2m1's widest step, and the rounding of the
// scale; typically a twelfth): after five, 2^-12 of it (typically 2^-18). So a pair has five columns, whose products
// are added in fp32 with the weights 8^-i.
// s is one for a column's whole length, since the products add up along it. It brings the row's largest value to [2^8, 2^9),
// in the range of e4m3 scales. Five terms are enough while the row's values lie near one another: a block whose largest is
// 11 binary orders below the row's still has normal scales for its last terms, and what a large value leaves, 2^-18 of it,
// is little against its neighbours. A row with some eight (h: sixteen) neighbours that lie lower, by an outlier, say, is
// multiplied in several passes: each takes what the passes before it left, 2^13 times larger, in five terms again, and the
// results of all are added. Where no row of a task is like that, one pass does. (Four neighbours of h would be as low by
// chance where gates are large, with silu(gate) about 0 for half of them: with gates of N(0, 50) for every row.)
// With bf16 weights x is a column as it is, and h the sum of two bf16 columns (16 bits).
//
// Both kernels list the routed experts and their pairs (route()) and then work in roles:
//   warps 0..3   turn accumulators into h, or into the sums of out
//   warp 4       issues the weight loads of a ring of slots, each 128 bytes of 256 weight rows
//   warps 5, 6   issue the products, one tile of 128 rows each
//   warps 7..    bring a slot's columns of x or h to shared memory, two or three warps a slot
// gate_up walks persistently over (pairs of an expert, 128 gate rows and their up rows); where that leaves more than
// half of the SMs without work, a cluster of blocks shares out the length of a row. In down a cluster owns 256 rows
// of out and shares out the experts; each block adds up its experts in order. A cluster adds up its blocks in order.
// No atomics on values: the same arguments give the same bits. down starts on SMs that gate_up leaves or does
// not need, and loads weights until h is there. Every wait is bounded (MOE_ERR_TIMEOUT).
//
// Why so, and what it measured (both kernels, one GB300, weights from DRAM; 6782 GB/s is the copy bandwidth):
//   256 experts of 7168 x 1024, top-8, NVFP4:    32 tokens 296 us (2.0 GB, 6.8 TB/s), 1 token 28.8 us (99 MB, 3.4 TB/s)
//   128 experts of 4096 x 768, top-8, bf16:      5 tokens 103 us (0.67 GB, 6.5 TB/s)
//   16 experts of 2112 x 704, top-3, bf16:       61 tokens 39 us (143 MB, 3.7 TB/s)
// The tensor core takes weights as they are stored, so no instruction is spent on a weight: converting them in
// registers for mma.sync was bound by those instructions (620 us for the 32 tokens). What is left is the terms of x and
// h, whose work grows with the pairs of an expert: at four an expert, 64 experts of 4096 x 1024, 32 tokens take 91 us,
// at eight 122 us, the dispatch, products and combine 101 us; MoELayer changes over between them. The small
// cases are bound by latency: two kernels' starts, the list of pairs, the first weights, h and the sums.
#include <algorithm>
#include <cstdint>
#include <mutex>

#include <cooperative_groups.h>

#include "expert_rows.cuh"
#include "experts_launch.h"
#include "tcgen05.cuh"
#include "tensor_map.h"

namespace cg = cooperative_groups;

namespace moe {
namespace {

// A team of PER converters takes every kTurns'th slot, or every `stages`th where there are fewer: a slot that it waits
// for is then at most one round of the ring ahead of the last one it filled, so that the parity that it waits
// for can only stand for the right phase.
constexpr int kLoadWarp = 4, kMmaWarp = 5, kConvertWarp = 7, kTurns = 4;
template <int PER>
constexpr int kThreadsOf = (kConvertWarp + kTurns * PER) * 32;
constexpr int kRows = 256;                    // weight rows of a slot: two tiles of 128
constexpr int kColumns = 64;                  // columns of a group of pairs
constexpr int kTerms = 5;                     // columns of a pair, NVFP4
constexpr int kMaxStages = 5;
constexpr int kOrders = 13;                   // binary orders that five terms take off the largest value of a block at least
constexpr int kSpread = 11;                   // binary orders below the row's largest at which a row makes do with one pass
constexpr int kKept = 32;                     // tasks whose columns' magnitudes and passes are kept
constexpr int kMaxRanks = 8;
constexpr uint32_t kTmemScales = 4 * kColumns;  // after two accumulators of two tiles
constexpr uint32_t kTmemScaleSet = 64;          // of a slot, for each tile: its scales and the columns', 16 each
constexpr int max_stages(bool nvfp4) { return nvfp4 ? int((512 - kTmemScales) / kTmemScaleSet) : kMaxStages; }

template <bool NVFP4, bool DOWN>
struct Shape {
    static constexpr int kChunk = NVFP4 ? 256 : 64;              // values of k in a slot
    static constexpr int kGroup = NVFP4 ? kColumns / 16 * 3 : DOWN ? kColumns / 2 : kColumns;  // pairs of a group
    static constexpr uint32_t kA = kRows * 128, kB = kColumns * 128;
    static constexpr uint32_t kSfA = NVFP4 ? kRows * 16 : 0, kSfB = NVFP4 ? 128 * 16 : 0;
    static constexpr uint32_t kSlot = kA + kB + kSfA + kSfB;
    // first column of pair j
    static __device__ __forceinline__ int column(int j) { return NVFP4 ? j / 3 * 16 + j % 3 * kTerms : DOWN ? 2 * j : j; }
    // columns of n pairs, a multiple of 16
    static __device__ __forceinline__ int columns(int n) {
        return NVFP4 ? (n + 2) / 3 * 16 : ((DOWN ? 2 : 1) * n + 15) / 16 * 16;
    }
};

struct LayerArgs {
    FewTokens f;
    int stages, chunks;  // slots of the ring; slots of a weight row
    int row_bytes;       // of a weight row
    int blocks;          // 128-row blocks of a weight matrix
    int k;
    int summed;          // columns of sums: T in down, in gate_up the pairs of the one task of a cluster
};

// Workspace: h as fp32 [pairs][I] and for each 32 of it [pairs][4 ceil(I/128)] two bytes, the exponents of the largest
// magnitude (high) and of the least largest of 16 neighbours that is not zero, or 255 (NVFP4); or two bf16 parts
// [pairs][2][I].
__device__ __forceinline__ float* h_values(const FewTokens& a) { return static_cast<float*>(a.workspace); }
__host__ __device__ __forceinline__ int h_parts(int I) { return (I + 127) / 128 * 4; }
__device__ __forceinline__ uint16_t* h_range(const FewTokens& a) {
    return reinterpret_cast<uint16_t*>(h_values(a) + int64_t(a.T) * a.K * a.I);
}

// ---------------------------------------------------------------------------
// routing: the experts that some pair names, their pairs, and groups of these
// ---------------------------------------------------------------------------
struct Routing {
    int groups;
    uint16_t* list;     // pairs by expert, in order
    uint16_t* expert;   // [groups]
    uint16_t* first;    // [groups + 1] into list
};

__host__ __device__ __forceinline__ size_t routing_bytes(int pairs) {
    return (size_t(3) * pairs + 1 + 7) / 8 * 16;
}
// A stable counting sort of the pairs by expert, by all threads of a block: chunks of 32 pairs are counted at
// once by warps (match), the experts' prefix sums by threads. `scratch`: E bytes for each chunk, 4 for each pair, 2
// for each expert (less than a ring of slots), 16-byte aligned, free again afterwards. `report`: write bad ids to the
// status word.
template <int kThreads>
__device__ __forceinline__ Routing route(const FewTokens& a, uint8_t* smem, uint8_t* scratch, int group, bool report) {
    __shared__ int warp_sum[kThreads / 32], n_groups;
    const int pairs = a.T * a.K, chunks = (pairs + 31) / 32, E = a.E;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Routing r;
    r.list = reinterpret_cast<uint16_t*>(smem);
    r.expert = r.list + pairs;
    r.first = r.expert + pairs;
    uint8_t* table = scratch;  // [chunks][E]: pairs of the chunk that name e
    int16_t* ids = reinterpret_cast<int16_t*>(scratch + (size_t(chunks) * E + 15) / 16 * 16);
    uint16_t* rank = reinterpret_cast<uint16_t*>(ids + pairs);
    uint16_t* start = rank + pairs;
    for (int i = tid; i < (chunks * E + 15) / 16; i += kThreads) reinterpret_cast<uint4*>(table)[i] = make_uint4(0, 0, 0, 0);
    int mine = -1;  // the first id of a thread, on its way while the table is cleared
    if (tid < pairs) mine = __ldg(a.ids + tid);
    __syncthreads();
    for (int c = warp; c < chunks; c += kThreads / 32) {
        const int p = c * 32 + lane;
        int e = c == warp ? mine : p < pairs ? __ldg(a.ids + p) : -1;
        const bool ok = p < pairs && e >= 0 && e < E;
        if (p < pairs && !ok && e != -1 && report) set_status(a.status, MOE_ERR_BAD_EXPERT_ID);
        if (!ok) e = -1;
        const unsigned same = __match_any_sync(kFullMask, e);
        const int before = __popc(same & ((1u << lane) - 1));
        if (p < pairs) ids[p] = int16_t(e), rank[p] = uint16_t(before);
        if (ok && (same >> lane) == 1) table[c * E + e] = uint8_t(before + 1);  // the last of its kind
    }
    __syncthreads();
    // a thread's neighbouring experts: pairs (low half) and groups (high half) of those before
    const int per = (E + kThreads - 1) / kThreads;
    int sum = 0;
    for (int e = tid * per; e < min(E, (tid + 1) * per); e++) {
        int n = 0;
        for (int c = 0; c < chunks; c++) n += table[c * E + e];
        sum += n + ((n + group - 1) / group << 16);
    }
    int before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFullMask, before, o);
        if (lane >= o) before += u;
    }
    if (lane == 31) warp_sum[warp] = before;
    __syncthreads();
    before -= sum;
    int total = 0;
    for (int w = 0; w < kThreads / 32; w++) {
        if (w < warp) before += warp_sum[w];
        total += warp_sum[w];
    }
    for (int e = tid * per; e < min(E, (tid + 1) * per); e++) {
        const int first = before & 0xffff, g = before >> 16;
        start[e] = uint16_t(first);
        int n = 0;
        for (int c = 0; c < chunks; c++) n += table[c * E + e];
        for (int j = 0; j * group < n; j++) {
            r.expert[g + j] = uint16_t(e);
            r.first[g + j] = uint16_t(first + j * group);
        }
        before += n + ((n + group - 1) / group << 16);
    }
    if (tid == 0) r.first[total >> 16] = uint16_t(total & 0xffff), n_groups = total >> 16;
    __syncthreads();
    for (int p = tid; p < pairs; p += kThreads) {
        const int e = ids[p];
        if (e < 0) continue;
        int at = start[e] + rank[p];
        for (int c = 0; c < p / 32; c++) at += table[c * E + e];
        r.list[at] = uint16_t(p);
    }
    __syncthreads();
    r.groups = n_groups;
    return r;
}

// ---------------------------------------------------------------------------
// shared state and waits
// ---------------------------------------------------------------------------
struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], shifts_ready;
    uint32_t tmem;
    int dead;           // a wait gave up
    int passes[kKept];  // of task i, and 256 (i + 1)
};

// gate_up with NVFP4: exponents of the largest magnitude of x for the pairs of a task, and 255 minus those of the least largest
// of eight that is not zero. (down has shifts and passes of all its pairs at once.)
struct Ranges {
    int largest[kKept][kColumns / 16 * 3], least[kKept][kColumns / 16 * 3];
};
template <bool NVFP4, bool DOWN>
constexpr size_t static_bytes() { return sizeof(Shared) + (NVFP4 && !DOWN ? sizeof(Ranges) : 0); }

__device__ __forceinline__ bool wait_or_die(const LayerArgs& a, Shared* s, uint32_t bar, uint32_t parity) {
    if (mbar_wait(bar, parity)) return true;
    *const_cast<volatile int*>(&s->dead) = 1;
    set_status(a.f.status, MOE_ERR_TIMEOUT);
    return false;
}
__device__ __forceinline__ bool warp_wait_or_die(const LayerArgs& a, Shared* s, uint32_t bar, uint32_t parity) {
    return __all_sync(kFullMask, wait_or_die(a, s, bar, parity));
}

// The passes of the block's task `i`, which a converter tells when it begins the task; as read before (`seen`), or waited for:
// 0 when the wait gave up.
__device__ __forceinline__ int passes_seen(Shared* s, int i) {
    int n;
    asm volatile("ld.relaxed.cta.shared::cta.s32 %0, [%1];" : "=r"(n) : "r"(smem_addr(&s->passes[i % kKept])) : "memory");
    return n;
}
__device__ __forceinline__ int await_passes(const LayerArgs& a, Shared* s, int i, int seen) {
    if (seen >> 8 == i + 1) return seen & 255;
    const uint64_t t0 = global_ns();
    for (int polls = 0; polls < kWaitMinPolls || global_ns() - t0 <= kWaitLimitNs; polls++) {
        seen = passes_seen(s, i);
        if (seen >> 8 == i + 1) return seen & 255;
    }
    *const_cast<volatile int*>(&s->dead) = 1;
    set_status(a.f.status, MOE_ERR_TIMEOUT);
    return 0;
}

// The block's n-th task: a group of pairs and, in gate_up, a 128-row block.
struct Task {
    int e, block, first, n;  // expert, first 128-row block, first pair in the list, pairs
};

// One block's tasks and place.
template <bool DOWN>
struct Work {
    int index, step, count, block;  // down: groups index, index + step, ..; gate_up: (group, block) likewise
    int c0, c1;                     // the slots of a weight row that are this block's

    __device__ __forceinline__ Work(const LayerArgs& a, const Routing& r, int rank, int ranks) {
        index = DOWN ? rank : int(blockIdx.x) / ranks;
        step = DOWN ? ranks : int(gridDim.x) / ranks;
        count = DOWN ? r.groups : r.groups * a.blocks;
        block = DOWN ? int(blockIdx.x) / ranks * 2 : 0;
        c0 = DOWN ? 0 : a.chunks * rank / ranks;
        c1 = DOWN ? a.chunks : a.chunks * (rank + 1) / ranks;
    }
    __device__ __forceinline__ int tasks() const { return index < count ? (count - index + step - 1) / step : 0; }
    __device__ __forceinline__ Task task(const LayerArgs& a, const Routing& r, int i) const {
        const int t = index + i * step, g = DOWN ? t : t / a.blocks;
        return Task{r.expert[g], DOWN ? block : t % a.blocks, r.first[g], r.first[g + 1] - r.first[g]};
    }
};

// ---------------------------------------------------------------------------
// roles
// ---------------------------------------------------------------------------
template <bool NVFP4, bool DOWN>
__device__ __forceinline__ void load_role(const LayerArgs& a, Shared* s, const Routing& r, const Work<DOWN>& work,
                                          uint32_t slots, const CUtensorMap* map) {
    using S = Shape<NVFP4, DOWN>;
    const uint8_t* sf = DOWN ? a.f.w2_sf : a.f.w13_sf;
    const int k64 = a.k / 64, tasks = work.tasks();
    int st = 0;
    uint32_t ph = 0;
    for (int i = 0; i < tasks; i++) {
        const Task t = work.task(a, r, i);
        for (int pass = 0, passes = 1; pass < passes; pass++) {
            for (int c = work.c0; c < work.c1; c++) {
                if (!wait_or_die(a, s, smem_addr(&s->empty[st]), ph ^ 1)) return;
                const uint32_t bar = smem_addr(&s->full[st]), slot = slots + st * S::kSlot;
                const bool second = !DOWN || t.block + 1 < a.blocks;
                const int q = NVFP4 ? min(4, k64 - 4 * c) : 0;
                mbar_expect_tx(bar, S::kA + q * 512 * (second ? 2 : 1));
                // dimensions (k, row, half, expert): 128 rows of both halves, or 256 rows
                tma_load_4d(slot, map, c * 128, t.block * 128, 0, t.e, bar);
                if (NVFP4) {
                    const int64_t block = DOWN ? int64_t(t.e) * a.blocks + t.block : int64_t(t.e) * 2 * a.blocks + t.block;
                    const uint32_t to = slot + S::kA + S::kB;
                    bulk_load_announced(to, sf + (block * k64 + 4 * c) * 512, q * 512, bar);
                    if (second)
                        bulk_load_announced(to + S::kSfA / 2,
                                            sf + ((block + (DOWN ? 1 : a.blocks)) * k64 + 4 * c) * 512, q * 512, bar);
                }
                if (++st == a.stages) st = 0, ph ^= 1;
            }
            if (NVFP4 && pass == 0 && (passes = await_passes(a, s, i, 0)) == 0) return;
        }
    }
}

// What the products of a tile read in the first slot; a slot further, kSlot / 16 more.
struct Operands {
    uint64_t a, b, sfa, sfb;
};

// The products of a slot's tile, 32 bytes of a row each (64 NVFP4 or 16 bf16 values), `q` of them.
template <bool NVFP4>
__device__ __forceinline__ void multiply_slot(const Operands& o, uint32_t off, uint32_t d, uint32_t ts, uint32_t idesc, int q,
                                              bool add) {
    if (NVFP4) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
            if (j >= q) break;
            tc_copy_scales(ts + j * 4, o.sfa + off + j * 32);
            tc_copy_scales(ts + 16 + j * 4, o.sfb + off + j * 32);
        }
    }
#pragma unroll
    for (int j = 0; j < 4; j++) {
        if (j >= q) break;
        if (NVFP4)
            tc_mma_nvfp4(d, o.a + off + 2 * j, o.b + off + 2 * j, idesc, ts + j * 4, ts + 16 + j * 4, add || j > 0);
        else
            tc_mma_bf16(d, o.a + off + 2 * j, o.b + off + 2 * j, idesc, add || j > 0);
    }
}

// A whole warp, for tile `half` of every slot; one lane issues. A slot costs the warp some hundred cycles beside its
// products, so what does not change from slot to slot is made before.
template <bool NVFP4, bool DOWN>
__device__ __forceinline__ void mma_role(const LayerArgs& a, Shared* s, const Routing& r, const Work<DOWN>& work,
                                         uint32_t slots, int half) {
    using S = Shape<NVFP4, DOWN>;
    const int tasks = work.tasks();
    const bool leader = elect_one();
    const uint32_t sf = slots + S::kA + S::kB;
    const Operands o{desc_k128(slots + half * (S::kA / 2)), desc_k128(slots + S::kA), desc_scales(sf + half * (S::kSfA / 2)),
                     desc_scales(sf + S::kSfA)};
    const uint32_t tmem = s->tmem, scales = tmem + kTmemScales + half * 32;
    const uint32_t full = smem_addr(s->full), empty = smem_addr(s->empty);
    const int q_last = (a.row_bytes - (a.chunks - 1) * 128) / 32;
    int st = 0, n_pass = 0;  // n_pass: passes of all tasks so far
    uint32_t ph = 0;
    for (int i = 0; i < tasks; i++) {
        const Task t = work.task(a, r, i);
        const int n = S::columns(t.n);
        const uint32_t idesc = NVFP4 ? idesc_nvfp4(n) : idesc_bf16(n);
        const bool there = !DOWN || t.block + half < a.blocks;
        for (int pass = 0, passes = 1; pass < passes; pass++, n_pass++) {
            const int buf = n_pass & 1;
            const uint32_t d = tmem + (buf * 2 + half) * kColumns;
            int seen = 0;
            if (!warp_wait_or_die(a, s, smem_addr(&s->acc_empty[buf]), (n_pass >> 1 & 1) ^ 1)) return;
            tc_fence_after();
            for (int c = work.c0; c < work.c1; c++) {
                if (!warp_wait_or_die(a, s, full + 8 * st, ph)) return;
                tc_fence_after();
                if (NVFP4 && c == work.c0) seen = passes_seen(s, i);
                if (leader) {
                    const uint32_t off = st * (S::kSlot / 16), ts = scales + st * kTmemScaleSet;
                    if (there) {
                        if (c + 1 < a.chunks || q_last == 4)
                            multiply_slot<NVFP4>(o, off, d, ts, idesc, 4, c > work.c0);
                        else
                            multiply_slot<NVFP4>(o, off, d, ts, idesc, q_last, c > work.c0);
                    }
                    tc_commit(empty + 8 * st);
                    if (c + 1 == work.c1) tc_commit(smem_addr(&s->acc_full[buf]));
                }
                __syncwarp();
                if (++st == a.stages) st = 0, ph ^= 1;
            }
            if (NVFP4 && pass == 0 && (passes = __reduce_min_sync(kFullMask, await_passes(a, s, i, seen))) == 0) return;
        }
    }
    // the last slot's arrival is the last that is on its way to this block's memory
    if (tasks > 0) warp_wait_or_die(a, s, empty + 8 * (st == 0 ? a.stages - 1 : st - 1), st == 0 ? ph ^ 1 : ph);
}

// 2^e as fp32, e in [-126, 127]
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// The power of two that brings a row's largest magnitude, by its (biased) exponent, to [2^8, 2^9); at most 2^126, with which
// a row below 2^-118 is left with what binary32 has of it.
constexpr int kMostShift = 126;
__device__ __forceinline__ int shift_of(int exponent) { return min(8 + 127 - exponent, kMostShift); }
// That of a pass.
__device__ __forceinline__ int pass_shift(int shift, int pass) { return min(shift + kOrders * pass, kMostShift); }
// The passes after the first that a row with shift `shift` needs, by the exponent of the least magnitude that counts.
__device__ __forceinline__ int more_passes(int shift, int exponent) {
    return max(8 + 127 - shift - exponent - kSpread + kOrders - 1, 0) / kOrders;
}
// A pass that comes before any that finds something of a block with this largest magnitude: the last term's scale is 0 where
// the block's largest is 2^-20 or less in the pass. (In the first pass it may be too small for binary32.)
__device__ __forceinline__ int first_pass(int shift, float block) {
    const int below = 8 - shift - (int(__float_as_uint(block) >> 23) - 127);
    return max(below - 29, 0) / kOrders;
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t min_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// The largest magnitude of eight bf16 values, twice.
__device__ __forceinline__ uint32_t largest_of(const uint4& w) {
    const uint32_t m =
        max_bf16x2(max_bf16x2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), max_bf16x2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
    return max_bf16x2(m, __byte_perm(m, m, 0x1032));
}

// Byte offset of 16-byte piece `piece` of row `row` in the 128-byte swizzle.
__device__ __forceinline__ uint32_t swizzled(int row, int piece) { return row * 128 + ((piece ^ (row & 7)) << 4); }

// Two fp32 values at once.
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
    uint64_t p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
    return p;
}
__device__ __forceinline__ float2 values_of(uint64_t p) {
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(p));
    return v;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t p;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(a), "l"(b));
    return p;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t p;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p) : "l"(a), "l"(b), "l"(c));
    return p;
}

// Term i of what is left of a block of 16 values: its codes, the scale, and in f what is left after it (`last`: nothing
// looks at that). The scale is that of 8^i f.
__device__ __forceinline__ uint2 split_term(uint64_t (&f)[8], int i, uint32_t* sf, bool last) {
    const float up = pow2(3 * i), down = pow2(-3 * i);
    float m[8];  // by halves: a chain of 16 is in the way of the next term
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const float2 v = values_of(f[j]);
        m[j] = fmaxf(fabsf(v.x), fabsf(v.y));
    }
#pragma unroll
    for (int h = 4; h; h /= 2)
#pragma unroll
        for (int j = 0; j < 4; j++)
            if (j < h) m[j] = fmaxf(m[j], m[j + h]);
    *sf = e4m3x2(m[0] * (up * (1.0f / 6.0f)), 0.0f) & 0xffu;
    const float s = e4m3_value(*sf) * down;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    r = s > 0.0f ? r : 0.0f;
    const uint64_t r2 = pair_of(r, r), s2 = pair_of(-s, -s);
    uint32_t q[2];
#pragma unroll
    for (int w = 0; w < 2; w++) {
        uint64_t* v = f + 4 * w;
        const float2 y0 = values_of(mul2(v[0], r2)), y1 = values_of(mul2(v[1], r2)), y2 = values_of(mul2(v[2], r2)),
                     y3 = values_of(mul2(v[3], r2));
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
            "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
            : "=r"(q[w])
            : "f"(y0.x), "f"(y0.y), "f"(y1.x), "f"(y1.y), "f"(y2.x), "f"(y2.y), "f"(y3.x), "f"(y3.y));
        if (last) continue;
        uint32_t h[4];
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
            "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
            "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
            "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
            : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
            : "r"(q[w]));
        // the product is exact, and the remainder as exact as fp32 gets
#pragma unroll
        for (int j = 0; j < 4; j++)
            v[j] = fma2(s2, pair_of(__half2float(__ushort_as_half(uint16_t(h[j]))),
                                    __half2float(__ushort_as_half(uint16_t(h[j] >> 16)))), v[j]);
    }
    return make_uint2(q[0], q[1]);
}

// 16 neighbouring values of x (bf16) or h (fp32) as they are in memory.
template <bool DOWN>
struct Sixteen {
    uint4 w[DOWN ? 4 : 2];

    __device__ __forceinline__ void load(const LayerArgs& a, int p, int k, bool ok) {
        const uint4* from = DOWN ? reinterpret_cast<const uint4*>(h_values(a.f) + int64_t(p) * a.k + k)
                                 : reinterpret_cast<const uint4*>(a.f.x + int64_t(p / a.f.K) * a.k + k);
#pragma unroll
        for (int l = 0; l < (DOWN ? 4 : 2); l++) {
            w[l] = make_uint4(0, 0, 0, 0);
            if (ok) w[l] = DOWN ? from[l] : __ldg(from + l);
        }
    }
    __device__ __forceinline__ float largest() const {
        if constexpr (DOWN) {
            float m = 0.0f;
#pragma unroll
            for (int l = 0; l < 4; l++)
                m = fmaxf(m, fmaxf(fmaxf(fabsf(__uint_as_float(w[l].x)), fabsf(__uint_as_float(w[l].y))),
                                   fmaxf(fabsf(__uint_as_float(w[l].z)), fabsf(__uint_as_float(w[l].w)))));
            return m;
        } else {
            return bf16_hi(max_bf16x2(largest_of(w[0]), largest_of(w[1])));
        }
    }
    __device__ __forceinline__ void scaled(float scale, uint64_t (&f)[8]) const {
        float v[16];
        if constexpr (DOWN) {
#pragma unroll
            for (int l = 0; l < 4; l++) {
                v[4 * l] = __uint_as_float(w[l].x), v[4 * l + 1] = __uint_as_float(w[l].y);
                v[4 * l + 2] = __uint_as_float(w[l].z), v[4 * l + 3] = __uint_as_float(w[l].w);
            }
        } else {
            unpack8(w[0], v);
            unpack8(w[1], v + 8);
        }
#pragma unroll
        for (int l = 0; l < 8; l++) f[l] = mul2(pair_of(v[2 * l], v[2 * l + 1]), pair_of(scale, scale));
    }
};

// A term of a block of 16 in row `row` of a slot's columns.
__device__ __forceinline__ void store_term(uint32_t to, int row, int block, uint2 q, uint32_t sf) {
    constexpr uint32_t kSf = Shape<true, false>::kB + Shape<true, false>::kSfA;
    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(to + swizzled(row, block >> 1) + (block & 1) * 8), "r"(q.x), "r"(q.y)
                 : "memory");
    asm volatile("st.shared.u8 [%0], %1;" ::"r"(to + kSf + (block >> 2) * 512 + (row % 32) * 16 + row / 32 * 4 + (block & 3)),
                 "r"(sf)
                 : "memory");
}

// The shift of pair j of the block's task i, and the passes after the first that its row needs.
template <bool DOWN>
__device__ __forceinline__ int row_shift(const Ranges* ranges, const int8_t* shifts, const Task& t, int i, int j) {
    return DOWN ? shifts[t.first + j] : shift_of(ranges->largest[i % kKept][j]);
}
template <bool DOWN>
__device__ __forceinline__ int row_more(const LayerArgs& a, const Ranges* ranges, const int8_t* shifts, const Task& t, int i,
                                        int j) {
    if (DOWN) return shifts[a.f.T * a.f.K + t.first + j];
    return more_passes(row_shift<DOWN>(ranges, shifts, t, i, j), 255 - ranges->least[i % kKept][j]);
}

// The further passes of task i, rarely: what the passes before leave, each block from its first pass on. The warp's place in
// the ring and its phase before, and after as st | ph << 8 | skip << 9; -1 when a wait gave up. Kept small: a kernel's start
// takes longer with its size. One token, which has no use for it, takes 28.1 us without it, 28.8 us with it, and 29.4 us with
// its terms unrolled or as a function of its own.
template <bool NVFP4, bool DOWN, int PER>
__device__ __forceinline__ int convert_more(const LayerArgs& a, Shared* s, const Ranges* ranges, const Routing& r,
                                            const Work<DOWN>& work, uint32_t slots, int v, const int8_t* shifts, int i,
                                            int passes, int st, int ph, int skip) {
    using S = Shape<NVFP4, DOWN>;
    const int lane = threadIdx.x & 31, turns = min(kTurns, a.stages), part = v % PER;
    const int block = lane % 16, pair = part * 2 + lane / 16;
    const Task t = work.task(a, r, i);
    for (int pass = 1; pass < passes; pass++) {
        int c = work.c0 + skip;
        for (; c < work.c1; c += turns) {
            if (!warp_wait_or_die(a, s, smem_addr(&s->empty[st]), ph ^ 1)) return -1;
            for (int j0 = 0; j0 + part * 2 < t.n; j0 += 2 * PER) {
                const int j = j0 + pair, at = min(j, t.n - 1), k = c * S::kChunk + block * 16;
                const int shift = row_shift<DOWN>(ranges, shifts, t, i, at);
                Sixteen<DOWN> now;
                now.load(a, r.list[t.first + at], k, k < a.k);
                int p = min(pass, first_pass(shift, now.largest()));
                uint64_t f[8];
                now.scaled(pass <= row_more<DOWN>(a, ranges, shifts, t, i, at) ? pow2(pass_shift(shift, p)) : 0.0f, f);
                const int row0 = S::column(at);
                for (;; p++) {
#pragma unroll 1
                    for (int l = 0; l < kTerms; l++) {
                        uint32_t sf;
                        const uint2 q = split_term(f, l, &sf, false);
                        if (p == pass && j < t.n) store_term(slots + st * S::kSlot + S::kA, row0 + l, block, q, sf);
                    }
                    if (p == pass) break;
                    const float up = pow2(pass_shift(shift, p + 1) - pass_shift(shift, p));
#pragma unroll
                    for (int l = 0; l < 8; l++) f[l] = mul2(f[l], pair_of(up, up));
                }
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&s->full[st]));
            st += turns;
            if (st >= a.stages) st -= a.stages, ph ^= 1;
        }
        skip = c - work.c1;
    }
    return st | ph << 8 | skip << 9;
}

// Warp `v` of the converters: its part of every `turns`th slot. down: `shifts` [pairs in the list], and behind them [pairs]
// the passes after the first that each needs.
template <bool NVFP4, bool DOWN, int PER>
__device__ __forceinline__ void convert_role(const LayerArgs& a, Shared* s, Ranges* ranges, const Routing& r,
                                             const Work<DOWN>& work, uint32_t slots, int v, int8_t* shifts) {
    using S = Shape<NVFP4, DOWN>;
    const int lane = threadIdx.x & 31, tasks = work.tasks();
    const int turns = min(kTurns, a.stages), turn = v / PER, part = v % PER;
    if (turn >= turns) return;
    int skip = turn, st = turn;  // slots of the next task before this warp's first one; its place in the ring
    uint32_t ph = 0;
    for (int i = 0; i < tasks; i++) {
        const Task t = work.task(a, r, i);
        const uint16_t* list = r.list + t.first;
        // NVFP4: a lane a block, a warp the sixteen blocks of two pairs, the slot's two warps every other two; the values
        // of the next pairs, or of the next slot's first, are on their way (the task's first ones while the largest are
        // looked for)
        const int block = lane % 16, pair = part * 2 + lane / 16;
        Sixteen<DOWN> now;
        auto load = [&](int c, int j) {
            const int k = c * S::kChunk + block * 16;
            const bool ok = c < work.c1 && j < t.n && k < a.k;
            now.load(a, list[ok ? j : 0], k, ok);
        };
        if (NVFP4) load(work.c0 + skip, pair);
        int passes = 1;
        int8_t* more = shifts + a.f.T * a.f.K;  // down: passes after the first
        auto shift_at = [&](int j) { return row_shift<DOWN>(ranges, shifts, t, i, j); };
        if (NVFP4 && DOWN && i == 0) {  // of every pair of the list, a thread a pair
            const int parts = h_parts(a.k);
            for (int at = v * 32 + lane; at < r.first[r.groups]; at += PER * turns * 32) {
                const uint2* from = reinterpret_cast<const uint2*>(h_range(a.f) + int64_t(r.list[at]) * parts);
                uint32_t most = 0, least = ~0u;  // of two halves
#pragma unroll 8
                for (int p = 0; p < parts / 4; p++) {
                    const uint2 w = from[p];
                    most = max_u16x2(most, max_u16x2(w.x, w.y));
                    least = min_u16x2(least, min_u16x2(w.x & 0x00ff00ffu, w.y & 0x00ff00ffu));
                }
                const int shift = shift_of(max(most & 0xffffu, most >> 16) >> 8);
                shifts[at] = int8_t(shift);
                more[at] = int8_t(more_passes(shift, min(least & 0xffffu, least >> 16)));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&s->shifts_ready));
            if (!warp_wait_or_die(a, s, smem_addr(&s->shifts_ready), 0)) return;
        }
        if (NVFP4 && !DOWN) {
            int *largest = ranges->largest[i % kKept], *lowest = ranges->least[i % kKept];
            // every warp looks at its part of the rows
            for (int j = 0; j < t.n; j++) {
                const uint16_t* x = a.f.x + int64_t(list[j] / a.f.K) * a.k;
                uint32_t most = 0, least = ~0u;  // a bf16 magnitude, twice; least: of those that are not zero, minus one
                for (int k0 = (v * 32 + lane) * 8; k0 < a.k; k0 += 4 * PER * turns * 256) {
                    uint4 w[4];
#pragma unroll
                    for (int u = 0; u < 4; u++) {
                        const int k = k0 + u * PER * turns * 256;
                        w[u] = k < a.k ? __ldg(reinterpret_cast<const uint4*>(x + k)) : make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int u = 0; u < 4; u++) {
                        const uint32_t m = largest_of(w[u]);
                        most = max(most, m), least = min(least, m - 1);
                    }
                }
                most = __reduce_max_sync(kFullMask, most), least = __reduce_min_sync(kFullMask, least);
                if (lane == 0) {
                    atomicMax(largest + j, int(most >> 23));
                    if (least != ~0u) atomicMax(lowest + j, 255 - int((least + 1) >> 23));
                }
            }
            // long done with: a converter is at most 8 tasks ahead of what turns accumulators into results
            if (v == 0 && lane < kColumns / 16 * 3)
                ranges->largest[(i + kKept / 2) % kKept][lane] = ranges->least[(i + kKept / 2) % kKept][lane] = 0;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&s->shifts_ready));
            if (!warp_wait_or_die(a, s, smem_addr(&s->shifts_ready), i & 1)) return;
        }
        if (NVFP4) {
            passes = 1 + __reduce_max_sync(kFullMask, lane < t.n ? row_more<DOWN>(a, ranges, shifts, t, i, lane) : 0);
            if (v == 0 && lane == 0)
                asm volatile("st.relaxed.cta.shared::cta.s32 [%0], %1;" ::"r"(smem_addr(&s->passes[i % kKept])),
                             "r"((i + 1) << 8 | passes)
                             : "memory");
        }
        int c = work.c0 + skip;
        for (; c < work.c1; c += turns) {
            const uint32_t to = slots + st * S::kSlot + S::kA;
            bool free = false;  // the slot: the first values are ready before it is waited for
            if (NVFP4) {
#pragma unroll 1
                for (int j0 = 0; j0 < t.n; j0 += 2 * PER) {
                    const int j = j0 + pair, at = min(j, t.n - 1);
                    uint64_t f[8];
                    now.scaled(pow2(shift_at(at)), f);
                    load(j0 + 2 * PER < t.n ? c : c + turns, j0 + 2 * PER < t.n ? j + 2 * PER : pair);
                    if (j0 + part * 2 >= t.n) continue;
                    uint2 q[kTerms];
                    uint32_t sf[kTerms];
#pragma unroll
                    for (int l = 0; l < kTerms; l++) q[l] = split_term(f, l, &sf[l], l + 1 == kTerms);
                    if (!free && !warp_wait_or_die(a, s, smem_addr(&s->empty[st]), ph ^ 1)) return;
                    free = true;
                    if (j >= t.n) continue;
                    const int row0 = S::column(j);
#pragma unroll
                    for (int l = 0; l < kTerms; l++) store_term(to, row0 + l, block, q[l], sf[l]);
                }
            } else {
                const int parts = DOWN ? 2 : 1;
                for (int u0 = part * 128; u0 < t.n * parts * 8; u0 += PER * 128) {  // pieces of 8 values: row u / 8, piece u % 8
                    uint4 w[4];
#pragma unroll
                    for (int l = 0; l < 4; l++) {
                        const int u = u0 + l * 32 + lane, row = u / 8, k = c * S::kChunk + u % 8 * 8;
                        w[l] = make_uint4(0, 0, 0, 0);
                        if (row < t.n * parts && k < a.k) {
                            const int p = list[row / parts];
                            const uint16_t* from =
                                DOWN ? static_cast<const uint16_t*>(a.f.workspace) + (int64_t(p) * 2 + row % 2) * a.k
                                     : a.f.x + int64_t(p / a.f.K) * a.k;
                            w[l] = *reinterpret_cast<const uint4*>(from + k);
                        }
                    }
                    if (!free && !warp_wait_or_die(a, s, smem_addr(&s->empty[st]), ph ^ 1)) return;
                    free = true;
#pragma unroll
                    for (int l = 0; l < 4; l++) {
                        const int u = u0 + l * 32 + lane, row = u / 8;
                        if (row < t.n * parts)
                            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to + swizzled(row, u % 8)),
                                         "r"(w[l].x), "r"(w[l].y), "r"(w[l].z), "r"(w[l].w)
                                         : "memory");
                    }
                }
            }
            if (!free && !warp_wait_or_die(a, s, smem_addr(&s->empty[st]), ph ^ 1)) return;
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&s->full[st]));
            st += turns;
            if (st >= a.stages) st -= a.stages, ph ^= 1;
        }
        skip = c - work.c1;
        if (NVFP4 && passes > 1) {
            const int next =
                convert_more<NVFP4, DOWN, PER>(a, s, ranges, r, work, slots, v, shifts, i, passes, st, int(ph), skip);
            if (next < 0) return;
            st = next & 0xff, ph = next >> 8 & 1, skip = next >> 9;
        }
    }
}

// Sums of a pair's columns, in v[16] from the pair's tile of 16 columns on.
template <bool NVFP4, bool DOWN>
__device__ __forceinline__ float pair_sum(const float* v, int j) {
    if (!NVFP4) return DOWN ? v[2 * j] + v[2 * j + 1] : v[j];
    float y = v[j * kTerms + kTerms - 1];
#pragma unroll
    for (int i = kTerms - 2; i >= 0; i--) y = fmaf(y, 0.125f, v[j * kTerms + i]);
    return y;
}

// h of row `row` and pair p from its gate and up sums; a warp's lanes have 32 neighbouring rows.
template <bool NVFP4>
__device__ __forceinline__ void store_h(const FewTokens& f, int p, int row, float gate, float up) {
    const float h = row < f.I ? swiglu(gate, up) : 0.0f;
    if (NVFP4) {
        if (row < f.I) h_values(f)[int64_t(p) * f.I + row] = h;
        float m = fabsf(h);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, o));
        const uint32_t most = __reduce_max_sync(kFullMask, __float_as_uint(m));
        const uint32_t least = __reduce_min_sync(kFullMask, __float_as_uint(m) - 1);
        if (row % 32 == 0)
            h_range(f)[int64_t(p) * h_parts(f.I) + row / 32] =
                uint16_t(most >> 23 << 8 | (least == ~0u ? 255u : (least + 1) >> 23));
    } else if (row < f.I) {
        uint16_t* to = static_cast<uint16_t*>(f.workspace) + int64_t(p) * 2 * f.I + row;
        const uint32_t hi = pack_bf16x2(h, 0.0f) & 0xffffu;
        to[0] = uint16_t(hi);
        to[f.I] = uint16_t(pack_bf16x2(h - bf16_lo(hi), 0.0f));
    }
}

// `sums` (of two rows, a thread's own): down's [T][kRows], or this block's [pairs][kRows] in the first block of a cluster
// of gate_up, which has one task together; null where gate_up's tasks are its own.
template <bool NVFP4, bool DOWN>
__device__ __forceinline__ void result_role(const LayerArgs& a, Shared* s, const Ranges* ranges, const Routing& r,
                                            const Work<DOWN>& work, float* sums, const int8_t* shifts) {
    using S = Shape<NVFP4, DOWN>;
    constexpr int kPairs = NVFP4 ? 3 : DOWN ? 8 : 16;  // pairs of 16 columns
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tasks = work.tasks();
    const uint32_t lanes = uint32_t(warp * 32) << 16;
    int n_pass = 0;  // passes of all tasks so far
    for (int i = 0; i < tasks; i++) {
        const Task t = work.task(a, r, i);
        const float* alphas = DOWN ? a.f.alpha2 : a.f.alpha13;
        const float alpha = alphas ? __ldg(alphas + t.e) : 1.0f;
        float earlier[2][NVFP4 && !DOWN ? S::kGroup : 1];  // sums of the passes before, where there are several
        for (int pass = 0, passes = 1; pass < passes; pass++, n_pass++) {
            const int buf = n_pass & 1;
            if (!warp_wait_or_die(a, s, smem_addr(&s->acc_full[buf]), n_pass >> 1 & 1)) return;
            tc_fence_after();
            const int seen = NVFP4 && pass == 0 ? passes_seen(s, i) : 0;
            if (NVFP4 && pass == 0 && (passes = __reduce_min_sync(kFullMask, await_passes(a, s, i, seen))) == 0) return;
            for (int j0 = 0, c = 0; j0 < t.n; j0 += kPairs, c += 16) {
                float v0[16], v1[16];
                tmem_load16(s->tmem + lanes + buf * 2 * kColumns + c, v0);
                tmem_load16(s->tmem + lanes + buf * 2 * kColumns + kColumns + c, v1);
                if (j0 + kPairs >= t.n) {  // the last columns: the accumulator is free
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&s->acc_empty[buf]));
                }
#pragma unroll
                for (int j = 0; j < kPairs; j++) {
                    if (j0 + j >= t.n) break;
                    const int p = r.list[t.first + j0 + j];
                    float y0 = pair_sum<NVFP4, DOWN>(v0, j) * alpha, y1 = pair_sum<NVFP4, DOWN>(v1, j) * alpha;
                    if (NVFP4) {
                        const float unscale = pow2(-pass_shift(row_shift<DOWN>(ranges, shifts, t, i, j0 + j), pass));
                        y0 *= unscale, y1 *= unscale;
                    }
                    if (DOWN) {
                        float* to = sums + (p / a.f.K) * kRows + warp * 32 + lane;
                        const float f = __ldg(a.f.w + p);
                        to[0] = fmaf(f, y0, to[0]);
                        to[128] = fmaf(f, y1, to[128]);
                    } else if (sums) {
                        float* to = sums + (j0 + j) * kRows + warp * 32 + lane;
                        to[0] = pass == 0 ? y0 : to[0] + y0;
                        to[128] = pass == 0 ? y1 : to[128] + y1;
                    } else {
                        if constexpr (NVFP4 && !DOWN) {
                            if (pass > 0) y0 += earlier[0][j0 + j], y1 += earlier[1][j0 + j];
                            if (pass + 1 < passes) {
                                earlier[0][j0 + j] = y0, earlier[1][j0 + j] = y1;
                                continue;
                            }
                        }
                        store_h<NVFP4>(a.f, p, t.block * 128 + warp * 32 + lane, y0, y1);
                    }
                }
            }
        }
    }
}

template <bool NVFP4, bool DOWN, int PER>
__global__ void __launch_bounds__(kThreadsOf<PER>, 1)
    few_tokens_kernel(const __grid_constant__ LayerArgs a, const __grid_constant__ CUtensorMap map) {
    using S = Shape<NVFP4, DOWN>;
    constexpr int kThreads = kThreadsOf<PER>;
    extern __shared__ uint8_t raw[];
    __shared__ Shared shared;
    Shared* s = &shared;
    Ranges* ranges = nullptr;
    if constexpr (NVFP4 && !DOWN) {
        __shared__ Ranges of_rows;
        ranges = &of_rows;
    }
    uint8_t* base = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);  // slots on swizzle atoms
    const uint32_t slots = smem_addr(base);
    const cg::cluster_group cluster = cg::this_cluster();
    const int rank = cluster.block_rank(), ranks = cluster.num_blocks();
    float* sums = reinterpret_cast<float*>(base + a.stages * S::kSlot);
    uint8_t* lists = base + a.stages * S::kSlot + sizeof(float) * kRows * a.summed * (DOWN ? 1 : ranks);
    int8_t* shifts = reinterpret_cast<int8_t*>(lists + routing_bytes(a.f.T * a.f.K));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == kMmaWarp) tmem_alloc(smem_addr(&s->tmem), 512);
    if (threadIdx.x == 0) {
        s->dead = 0;
        for (int i = 0; i < a.stages; i++) {
            mbar_init(smem_addr(&s->full[i]), 1 + PER);  // the loads' issuer and the converters
            mbar_init(smem_addr(&s->empty[i]), 2);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(smem_addr(&s->acc_full[i]), 2);
            mbar_init(smem_addr(&s->acc_empty[i]), 4);
        }
        mbar_init(smem_addr(&s->shifts_ready), PER * min(kTurns, a.stages));
        mbar_fence_init();
    }
    if (DOWN && warp < 4)
        for (int i = threadIdx.x; i < kRows * a.f.T; i += 128) sums[i] = 0.0f;  // a thread's own two rows
    if (NVFP4 && threadIdx.x < kKept) s->passes[threadIdx.x] = 0;
    if (NVFP4 && !DOWN)
        for (int i = threadIdx.x; i < kKept * (kColumns / 16 * 3); i += kThreads)
            ranges->largest[0][i] = ranges->least[0][i] = 0;
    // down is released once every block of gate_up has come past its own wait: what came before gate_up is done, and
    // only h, which the converters wait for, is not
    if (!DOWN) {
        pdl_wait();
        pdl_release();
        // the tokens' rows to L2, before the first weights: behind these they would wait for a whole ring of every SM
        const char* x = reinterpret_cast<const char*>(a.f.x);
        const int64_t at = (int64_t(blockIdx.x) * kThreads + threadIdx.x) * 128;
        if (at < int64_t(a.f.T) * a.f.H * 2) asm volatile("prefetch.global.L2 [%0];" ::"l"(x + at));
    }
    const Routing r = route<kThreads>(a.f, lists, base, S::kGroup, !DOWN && blockIdx.x == 0);
    const Work<DOWN> work(a, r, rank, ranks);
    fence_proxy_async();  // route()'s scratch is where the first loads land
    tc_fence_before();
    if (!DOWN && a.summed > 0)
        cluster.sync();  // the first block's shared memory is there
    else
        __syncthreads();
    tc_fence_after();

    if (warp < 4)
        result_role<NVFP4, DOWN>(a, s, ranges, r, work, a.summed == 0 ? nullptr
                                                : DOWN      ? sums
                                                            : cluster.map_shared_rank(sums, 0) + rank * a.summed * kRows,
                                 shifts);
    else if (warp == kLoadWarp) {
        if (lane == 0) load_role<NVFP4, DOWN>(a, s, r, work, slots, &map);
    } else if (warp < kConvertWarp) {
        mma_role<NVFP4, DOWN>(a, s, r, work, slots, warp - kMmaWarp);
    } else {
        if (DOWN) pdl_wait();
        convert_role<NVFP4, DOWN, PER>(a, s, ranges, r, work, slots, warp - kConvertWarp, shifts);
    }
    if (DOWN) pdl_wait();  // a block without work does not end before gate_up has either
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*const_cast<volatile int*>(&s->dead) && threadIdx.x == 0) {
        // whatever is still in flight lands in this block's memory: give it time before that is freed
        const uint64_t t0 = global_ns();
        while (global_ns() - t0 < kDrainLimitNs) __nanosleep(1000);
    }
    __syncthreads();
    if (warp == kMmaWarp) tmem_free(s->tmem, 512);
    if (a.summed == 0) return;
    cluster.sync();
    if (DOWN) {
        for (int i = rank * kThreads + int(threadIdx.x); i < kRows * a.f.T; i += ranks * kThreads) {
            const int row = work.block * 128 + i % kRows;
            float v[kMaxRanks], y = 0.0f;
#pragma unroll
            for (int b = 0; b < kMaxRanks; b++) v[b] = b < ranks ? cluster.map_shared_rank(sums, b)[i] : 0.0f;
#pragma unroll
            for (int b = 0; b < kMaxRanks; b++) y += v[b];
            if (row < a.f.H) a.f.out[int64_t(i / kRows) * a.f.H + row] = uint16_t(pack_bf16x2(y, 0.0f));
        }
    } else if (rank == 0 && work.tasks() > 0) {
        const Task t = work.task(a, r, 0);
        for (int i = threadIdx.x; i < 128 * t.n; i += kThreads) {
            const int j = i / 128, row = i % 128;
            float gate = 0.0f, up = 0.0f;
            for (int b = 0; b < ranks; b++) {
                const float* from = sums + (b * a.summed + j) * kRows + row;
                gate += from[0], up += from[128];
            }
            store_h<NVFP4>(a.f, r.list[t.first + j], t.block * 128 + row, gate, up);
        }
    }
    if (DOWN) cluster.sync();  // no block's sums go before the others have read them
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
// Whether `owners` clusters of `ranks` blocks can be resident at once (GPCs hold whole clusters), cached per
// device: it depends on the kernel, its shared memory and the device alone.
template <bool NVFP4, bool DOWN, int PER, typename Kernel>
bool clusters_fit(const LaunchCtx& ctx, Kernel kern, cudaLaunchConfig_t cfg, int owners, int ranks) {
    constexpr int kDevices = 64;
    static std::mutex mu;
    static struct {
        size_t smem;
        int most;
    } cache[kDevices][kMaxRanks + 1];
    const bool known = ctx.device >= 0 && ctx.device < kDevices;
    if (known) {
        std::lock_guard<std::mutex> lock(mu);
        const auto& c = cache[ctx.device][ranks];
        if (c.smem == cfg.dynamicSmemBytes) return owners <= c.most;
    }
    int most = 0;
    cfg.gridDim = dim3(unsigned(ranks));
    if (cudaOccupancyMaxActiveClusters(&most, kern, &cfg) != cudaSuccess) {
        cudaGetLastError();  // a size that the device does not have does not fit
        most = 0;
    }
    if (known) {
        std::lock_guard<std::mutex> lock(mu);
        cache[ctx.device][ranks].smem = cfg.dynamicSmemBytes;
        cache[ctx.device][ranks].most = most;
    }
    return owners <= most;
}

template <bool NVFP4, bool DOWN, int PER>
cudaError_t launch_half(const LaunchCtx& ctx, const FewTokens& f) {
    using S = Shape<NVFP4, DOWN>;
    constexpr size_t kMost = 226 * 1024;  // dynamic shared memory beside the static part
    auto kern = few_tokens_kernel<NVFP4, DOWN, PER>;
    // first: it makes the device's context current in a thread that has made no CUDA call yet, and the map needs one
    const cudaError_t err = allow_shared_memory(kern, kMost - static_bytes<NVFP4, DOWN>());
    if (err != cudaSuccess) return err;
    const int rows = DOWN ? f.H : f.I, k = DOWN ? f.I : f.H, pairs = f.T * f.K;
    LayerArgs a{f, 0, 0, NVFP4 ? k / 2 : 2 * k, (rows + 127) / 128, k, 0};
    a.chunks = (a.row_bytes + 127) / 128;

    CUtensorMap map;
    const uint64_t dims[4] = {uint64_t(a.row_bytes), uint64_t(rows), DOWN ? 1u : 2u, uint64_t(f.E)};
    const uint32_t box[4] = {128, DOWN ? 256u : 128u, DOWN ? 1u : 2u, 1};
    if (!make_map(&map, DOWN ? f.w2 : f.w13, 4, dims, box)) return cudaErrorInvalidValue;

    // gate_up: a cluster for each task while at least two blocks a task fit the SMs, else a block for each SM
    const int64_t tasks = int64_t(pairs) * a.blocks;
    const int64_t owners = DOWN ? (a.blocks + 1) / 2 : std::min<int64_t>(tasks, ctx.num_sms);
    int ranks = int(std::min<int64_t>({kMaxRanks, ctx.num_sms / owners, DOWN ? std::min(pairs, f.E) : a.chunks}));
    // whole pairs of SMs: with odd sizes, clusters that start as SMs become free did not all fit (a second
    // round of down, 28 clusters of 5: 459 us for 32 tokens against 345 us)
    ranks = ranks > 1 ? ranks / 2 * 2 : 1;
    const int task_pairs = std::min(pairs, S::kGroup);
    if (!DOWN) ranks = std::min(ranks, std::max(1, 32 / task_pairs / 2 * 2));  // their sums: at most 32 KB
    if (DOWN) a.summed = f.T;
    else if (ranks > 1) a.summed = task_pairs;
    const size_t fixed =
        1024 + sizeof(float) * kRows * a.summed * (DOWN ? 1 : ranks) + routing_bytes(pairs) + 2 * pairs;
    a.stages = int(std::min<size_t>(max_stages(NVFP4), (kMost - static_bytes<NVFP4, DOWN>() - fixed) / S::kSlot));

    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreadsOf<PER>);
    cfg.dynamicSmemBytes = fixed + size_t(a.stages) * S::kSlot;
    cfg.stream = ctx.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    for (;; ranks -= ranks > 2 ? 2 : 1) {
        attr[0].val.clusterDim.x = unsigned(ranks);
        if (ranks == 1 || clusters_fit<NVFP4, DOWN, PER>(ctx, kern, cfg, int(owners), ranks)) break;
    }
    cfg.gridDim = dim3(unsigned(owners * ranks));
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a, map);
}

}  // namespace

size_t few_tokens_workspace(int64_t T, int K, int, int I, int) {
    return size_t(T) * K * (size_t(I) * sizeof(float) + h_parts(I) * sizeof(uint16_t));
}

template <bool NVFP4, int PER>
static cudaError_t launch_layer(const LaunchCtx& ctx, const FewTokens& f) {
    const cudaError_t err = launch_half<NVFP4, false, PER>(ctx, f);
    return err != cudaSuccess ? err : launch_half<NVFP4, true, PER>(ctx, f);
}

// Three converters a slot from two pairs an expert on, two below and with bf16 weights, which are only copied: 64 experts
// of 4096 x 1024, top-8, 64 tokens 122 us with three, 131 with two and 128 with four (which have fewer registers); 256
// experts of 7168 x 1024, one token 27.5, 26.9 and 28.5 us (more warps start later), 32 tokens 296, 295 and 298 us.
cudaError_t launch_few_tokens(const LaunchCtx& ctx, const FewTokens& f) {
    if (!f.nvfp4) return launch_layer<false, 2>(ctx, f);
    return f.T * f.K > 2 * f.E ? launch_layer<true, 3>(ctx, f) : launch_layer<true, 2>(ctx, f);
}

}  // namespace moe
