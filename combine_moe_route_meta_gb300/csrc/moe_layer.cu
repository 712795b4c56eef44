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
//   r0 = x 2^s;  q_i = nvfp4(8^i r_i);  r_{i+1} = r_i - 8^-i q_i;   x 2^s ~ sum 8^-i q_i,
// each of which leaves at most a sixth of the block's largest value (typically a twelfth): after five, 2^-13 of
// it (typically 2^-18). So a pair has five columns, whose products are added in fp32 with the weights 8^-i.
// s, for each column's whole length, brings its largest value to [2^8, 2^9), in the range of e4m3 scales.
// With bf16 weights x is a column as it is, and h the sum of two bf16 columns (16 bits).
//
// Both kernels list the routed experts and their pairs (route()) and then work in roles:
//   warps 0..3   turn accumulators into h, or into the sums of out
//   warp 4       issues the weight loads of a ring of slots, each 128 bytes of 256 weight rows
//   warp 5       issues the products
//   warps 6..13  bring a slot's columns of x or h to shared memory, two warps a slot
// gate_up walks persistently over (pairs of an expert, 128 gate rows and their up rows). In down a cluster of
// blocks owns 256 rows of out and shares out the experts; each block adds up its experts in order, the cluster
// adds up the blocks in order. No atomics on values: the same arguments give the same bits. Every wait
// is bounded (MOE_ERR_TIMEOUT).
#include <algorithm>
#include <cstdint>

#include <cooperative_groups.h>

#include "expert_rows.cuh"
#include "experts_launch.h"
#include "tcgen05.cuh"
#include "tensor_map.h"

namespace cg = cooperative_groups;

namespace moe {
namespace {

// A pair of converters takes every kTurns'th slot, or every `stages`th where there are fewer: a slot that it waits
// for is then at most one round of the ring ahead of the last one it filled, so that the parity that it waits
// for can only stand for the right phase.
constexpr int kLoadWarp = 4, kMmaWarp = 5, kConvertWarp = 6, kTurns = 4, kConvertWarps = 2 * kTurns;
constexpr int kThreads = (kConvertWarp + kConvertWarps) * 32;
constexpr int kRows = 256;                    // weight rows of a slot: two tiles of 128
constexpr int kColumns = 64;                  // columns of a group of pairs
constexpr int kTerms = 5;                     // columns of a pair, NVFP4
constexpr int kMaxStages = 5;
constexpr int kShifts = 16;                   // tasks whose powers of two are kept
constexpr uint32_t kTmemScales = 4 * kColumns;  // after two accumulators of two tiles
constexpr uint32_t kTmemScaleSet = 48;          // two tiles' and the columns' scales of a slot, 16 each
static_assert(kTmemScales + kMaxStages * kTmemScaleSet <= 512, "tensor memory");

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
};

// Workspace: h as fp32 [pairs][I] and the largest magnitude of each 32 of it [pairs][I/32] (NVFP4), or
// two bf16 parts [pairs][2][I].
__device__ __forceinline__ float* h_values(const FewTokens& a) { return static_cast<float*>(a.workspace); }
__host__ __device__ __forceinline__ int h_parts(int I) { return (I + 31) / 32; }
__device__ __forceinline__ float* h_largest(const FewTokens& a) { return h_values(a) + int64_t(a.T) * a.K * a.I; }

// ---------------------------------------------------------------------------
// routing: the experts that some pair names, their pairs, and groups of these
// ---------------------------------------------------------------------------
struct Routing {
    int groups;
    uint16_t* list;     // pairs by expert, in order
    uint16_t* expert;   // [groups]
    uint16_t* first;    // [groups + 1] into list
};

__host__ __device__ __forceinline__ size_t routing_bytes(int pairs, int E) {
    return (size_t(5) * pairs + 1 + size_t(2) * E + 7) / 8 * 16;
}

// All threads of a block; ends with a barrier. `report`: write bad ids to the status word.
__device__ __forceinline__ Routing route(const FewTokens& a, uint8_t* smem, int group, bool report) {
    __shared__ int n_groups;
    const int pairs = a.T * a.K, lane = threadIdx.x & 31;
    Routing r;
    int16_t* ids = reinterpret_cast<int16_t*>(smem);
    r.expert = reinterpret_cast<uint16_t*>(ids + pairs);  // first the experts in the order of their first pairs
    r.first = r.expert + pairs;
    r.list = r.first + pairs + 1;
    uint16_t* rank = r.list + pairs;
    uint16_t* count = rank + pairs;
    uint16_t* start = count + a.E;
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) count[e] = 0;
    for (int p = threadIdx.x; p < pairs; p += blockDim.x) {
        const int e = __ldg(a.ids + p);
        const bool ok = e >= 0 && e < a.E;
        if (!ok && e != -1 && report) set_status(a.status, MOE_ERR_BAD_EXPERT_ID);
        ids[p] = int16_t(ok ? e : -1);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const unsigned below = (1u << lane) - 1;
        int n = 0;
        for (int p0 = 0; p0 < pairs; p0 += 32) {
            const int p = p0 + lane, e = p < pairs ? ids[p] : -1;
            const unsigned same = __match_any_sync(kFullMask, e);
            const int before = e >= 0 ? count[e] + __popc(same & below) : 1;
            const unsigned firsts = __ballot_sync(kFullMask, before == 0);
            if (before == 0) r.expert[n + __popc(firsts & below)] = uint16_t(e);
            if (p < pairs) rank[p] = uint16_t(before);
            __syncwarp();
            if (e >= 0 && (same >> lane) == 1) count[e] = uint16_t(before + 1);  // the last of its kind
            n += __popc(firsts);
            __syncwarp();
        }
        // prefix sums of the experts' pairs and groups; the groups are written from the last experts to the
        // first, so that the list of experts that they take the place of is read before
        int pairs_before = 0, groups_before = 0;
        for (int i0 = 0; i0 < n; i0 += 32) {
            const int i = i0 + lane, c = i < n ? count[r.expert[i]] : 0;
            int v = c, u = (c + group - 1) / group;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v1 = __shfl_up_sync(kFullMask, v, o), u1 = __shfl_up_sync(kFullMask, u, o);
                if (lane >= o) v += v1, u += u1;
            }
            if (i < n) {
                start[r.expert[i]] = uint16_t(pairs_before + v - c);
                r.first[i] = uint16_t(groups_before + u - (c + group - 1) / group);  // its first group, for now
            }
            pairs_before += __shfl_sync(kFullMask, v, 31);
            groups_before += __shfl_sync(kFullMask, u, 31);
        }
        for (int i0 = (n - 1) / 32 * 32; i0 >= 0 && n > 0; i0 -= 32) {
            const int i = i0 + lane;
            const int e = i < n ? r.expert[i] : 0, c = i < n ? count[e] : 0, g0 = i < n ? r.first[i] : 0;
            __syncwarp();
            for (int g = 0; g * group < c; g++) {
                r.expert[g0 + g] = uint16_t(e);
                r.first[g0 + g] = uint16_t(start[e] + g * group);
            }
            __syncwarp();
        }
        if (lane == 0) r.first[groups_before] = uint16_t(pairs_before), n_groups = groups_before;
    }
    __syncthreads();
    for (int p = threadIdx.x; p < pairs; p += blockDim.x)
        if (ids[p] >= 0) r.list[start[ids[p]] + rank[p]] = uint16_t(p);
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
    int dead;  // a wait gave up
    int8_t shift[kShifts][kColumns];
};

__device__ __forceinline__ bool wait_or_die(const LayerArgs& a, Shared* s, uint64_t* bar, uint32_t parity) {
    if (mbar_wait(smem_addr(bar), parity)) return true;
    *const_cast<volatile int*>(&s->dead) = 1;
    set_status(a.f.status, MOE_ERR_TIMEOUT);
    return false;
}
__device__ __forceinline__ bool warp_wait_or_die(const LayerArgs& a, Shared* s, uint64_t* bar, uint32_t parity) {
    return __all_sync(kFullMask, wait_or_die(a, s, bar, parity));
}

// The block's n-th task: a group of pairs and, in gate_up, a 128-row block.
struct Task {
    int e, block, first, n;  // expert, first 128-row block, first pair in the list, pairs
};

// One block's tasks and place.
template <bool DOWN>
struct Work {
    int index, step, count, block;  // down: groups index, index + step, ..; gate_up: (group, block) likewise

    __device__ __forceinline__ Work(const LayerArgs& a, const Routing& r, int rank, int ranks) {
        index = DOWN ? rank : int(blockIdx.x);
        step = DOWN ? ranks : int(gridDim.x);
        count = DOWN ? r.groups : r.groups * a.blocks;
        block = DOWN ? int(blockIdx.x) / ranks * 2 : 0;
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
        for (int c = 0; c < a.chunks; c++) {
            if (!wait_or_die(a, s, &s->empty[st], ph ^ 1)) return;
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
    }
}

// The products of a slot, 32 bytes of a row each: 64 NVFP4 or 16 bf16 values.
template <bool NVFP4, bool DOWN>
__device__ __forceinline__ void multiply_slot(uint32_t slot, uint32_t d, uint32_t ts, uint32_t idesc, int q, bool second,
                                              bool add) {
    using S = Shape<NVFP4, DOWN>;
    const uint64_t a0 = desc_k128(slot), a1 = desc_k128(slot + S::kA / 2), b = desc_k128(slot + S::kA);
    if (NVFP4) {
        const uint32_t sf = slot + S::kA + S::kB;
        const uint64_t s0 = desc_scales(sf), s1 = desc_scales(sf + S::kSfA / 2), sb = desc_scales(sf + S::kSfA);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            if (j >= q) break;
            tc_copy_scales(ts + j * 4, s0 + j * 32);
            tc_copy_scales(ts + 16 + j * 4, s1 + j * 32);
            tc_copy_scales(ts + 32 + j * 4, sb + j * 32);
        }
    }
#pragma unroll
    for (int t = 0; t < 2; t++) {
        if (t == 1 && !second) break;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            if (j >= q) break;
            if (NVFP4)
                tc_mma_nvfp4(d + t * kColumns, (t ? a1 : a0) + 2 * j, b + 2 * j, idesc, ts + t * 16 + j * 4,
                             ts + 32 + j * 4, add || j > 0);
            else
                tc_mma_bf16(d + t * kColumns, (t ? a1 : a0) + 2 * j, b + 2 * j, idesc, add || j > 0);
        }
    }
}

// A whole warp; one lane issues.
template <bool NVFP4, bool DOWN>
__device__ __forceinline__ void mma_role(const LayerArgs& a, Shared* s, const Routing& r, const Work<DOWN>& work,
                                         uint32_t slots) {
    using S = Shape<NVFP4, DOWN>;
    const int tasks = work.tasks();
    const bool leader = elect_one();
    const uint32_t tmem = s->tmem;
    int st = 0;
    uint32_t ph = 0;
    for (int i = 0; i < tasks; i++) {
        const Task t = work.task(a, r, i);
        const int buf = i & 1, n = S::columns(t.n);
        const uint32_t d = tmem + buf * 2 * kColumns;
        const uint32_t idesc = NVFP4 ? idesc_nvfp4(n) : idesc_bf16(n);
        const bool second = !DOWN || t.block + 1 < a.blocks;
        if (!warp_wait_or_die(a, s, &s->acc_empty[buf], (i >> 1 & 1) ^ 1)) return;
        tc_fence_after();
        for (int c = 0; c < a.chunks; c++) {
            if (!warp_wait_or_die(a, s, &s->full[st], ph)) return;
            tc_fence_after();
            const int q = min(4, (a.row_bytes - c * 128) / 32);
            if (leader) {
                multiply_slot<NVFP4, DOWN>(slots + st * S::kSlot, d, tmem + kTmemScales + st * kTmemScaleSet, idesc, q,
                                           second, c > 0);
                tc_commit(smem_addr(&s->empty[st]));
                if (c + 1 == a.chunks) tc_commit(smem_addr(&s->acc_full[buf]));
            }
            __syncwarp();
            if (++st == a.stages) st = 0, ph ^= 1;
        }
    }
    // the last slot's arrival is the last that is on its way to this block's memory
    if (tasks > 0) warp_wait_or_die(a, s, &s->empty[st == 0 ? a.stages - 1 : st - 1], st == 0 ? ph ^ 1 : ph);
}

// 2^e as fp32, e in [-126, 127]
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// The power of two that brings a largest magnitude to [2^8, 2^9).
__device__ __forceinline__ int shift_of(float largest) {
    return largest == 0.0f ? 0 : 8 - max(int(__float_as_uint(largest) >> 23) - 127, -110);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFullMask, v, o));
    return v;
}

// Byte offset of 16-byte piece `piece` of row `row` in the 128-byte swizzle.
__device__ __forceinline__ uint32_t swizzled(int row, int piece) { return row * 128 + ((piece ^ (row & 7)) << 4); }

__device__ __forceinline__ void st_shared_v2(uint32_t at, uint32_t x, uint32_t y) {
    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(x), "r"(y) : "memory");
}

// A block of 16 values as the sum of kTerms NVFP4 blocks: codes to q[i], their scales to sf[i].
__device__ __forceinline__ void split16(float* f, uint2* q, uint32_t* sf) {
#pragma unroll
    for (int i = 0; i < kTerms; i++) {
        float amax = 0.0f;
#pragma unroll
        for (int j = 0; j < 16; j++) amax = fmaxf(amax, fabsf(f[j]));
        sf[i] = e4m3x2(amax * (1.0f / 6.0f), 0.0f) & 0xffu;
        const float s = e4m3_value(sf[i]);
        const float r = s > 0.0f ? __frcp_rn(s) : 0.0f;
        uint32_t b[8];
#pragma unroll
        for (int p = 0; p < 8; p++) b[p] = e2m1x2(f[2 * p] * r, f[2 * p + 1] * r);
        q[i] = make_uint2(b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24, b[4] | b[5] << 8 | b[6] << 16 | b[7] << 24);
        if (i + 1 < kTerms) {
            uint32_t s2, v[8];
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s2) : "h"(uint16_t(sf[i] * 0x101u)));
            decode8(q[i].x, s2, v);  // exact
            decode8(q[i].y, s2, v + 4);
#pragma unroll
            for (int p = 0; p < 8; p++) {
                f[2 * p] = 8.0f * (f[2 * p] - __half2float(__ushort_as_half(uint16_t(v[p]))));
                f[2 * p + 1] = 8.0f * (f[2 * p + 1] - __half2float(__ushort_as_half(uint16_t(v[p] >> 16))));
            }
        }
    }
}

// Warp `v` of the converters: half the work of every `turns`th slot.
template <bool NVFP4, bool DOWN>
__device__ __forceinline__ void convert_role(const LayerArgs& a, Shared* s, const Routing& r, const Work<DOWN>& work,
                                             uint32_t slots, int v) {
    using S = Shape<NVFP4, DOWN>;
    const int lane = threadIdx.x & 31, tasks = work.tasks();
    const int turns = min(kTurns, a.stages), turn = v / 2, half = v % 2;
    if (turn >= turns) return;
    int seq = 0, st = 0;  // slots so far, over all tasks; their place in the ring
    uint32_t ph = 0;
    for (int i = 0; i < tasks; i++) {
        const Task t = work.task(a, r, i);
        const uint16_t* list = r.list + t.first;
        if (NVFP4) {
            int8_t* shift = s->shift[i % kShifts];
            for (int j = v; j < t.n; j += 2 * turns) {
                float m = 0.0f;
                if (DOWN) {
                    const int parts = h_parts(a.k);
                    const float* from = h_largest(a.f) + int64_t(list[j]) * parts;
                    for (int p = lane; p < parts; p += 32) m = fmaxf(m, __ldg(from + p));
                } else {
                    const uint16_t* x = a.f.x + int64_t(list[j] / a.f.K) * a.k;
#pragma unroll 4
                    for (int k = lane * 8; k < a.k; k += 256) {
                        float f[8];
                        unpack8(__ldg(reinterpret_cast<const uint4*>(x + k)), f);
#pragma unroll
                        for (int l = 0; l < 8; l++) m = fmaxf(m, fabsf(f[l]));
                    }
                }
                const int sh = shift_of(warp_max(m));
                if (lane == 0) shift[j] = int8_t(sh);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&s->shifts_ready));
            if (!warp_wait_or_die(a, s, &s->shifts_ready, i & 1)) return;
        }
        for (int c = 0; c < a.chunks; c++, seq++) {
            if (seq % turns == turn) {
                const uint32_t to = slots + st * S::kSlot + S::kA;
                bool free = false;  // the slot: the first values are ready before it is waited for
                if (NVFP4) {
                    const uint32_t sf_to = to + S::kB + S::kSfA;
                    for (int u0 = half * 32; u0 < t.n * 16; u0 += 64) {  // blocks of 16: pair u / 16, block u % 16 of the slot
                        const int u = u0 + lane, j = u / 16, b = u % 16, k = c * S::kChunk + b * 16;
                        float f[16];
#pragma unroll
                        for (int l = 0; l < 16; l++) f[l] = 0.0f;
                        if (j < t.n && k < a.k) {
                            if (DOWN) {
                                const float4* h = reinterpret_cast<const float4*>(h_values(a.f) + int64_t(list[j]) * a.k + k);
#pragma unroll
                                for (int l = 0; l < 4; l++) {
                                    const float4 w = __ldg(h + l);
                                    f[4 * l] = w.x, f[4 * l + 1] = w.y, f[4 * l + 2] = w.z, f[4 * l + 3] = w.w;
                                }
                            } else {
                                const uint4* x = reinterpret_cast<const uint4*>(a.f.x + int64_t(list[j] / a.f.K) * a.k + k);
                                unpack8(__ldg(x), f);
                                unpack8(__ldg(x + 1), f + 8);
                            }
                            const float scale = pow2(s->shift[i % kShifts][j]);
#pragma unroll
                            for (int l = 0; l < 16; l++) f[l] *= scale;
                        }
                        uint2 q[kTerms];
                        uint32_t sf[kTerms];
                        split16(f, q, sf);
                        if (!free && !warp_wait_or_die(a, s, &s->empty[st], ph ^ 1)) return;
                        free = true;
                        if (j < t.n) {
#pragma unroll
                            for (int l = 0; l < kTerms; l++) {
                                const int row = S::column(j) + l;
                                st_shared_v2(to + swizzled(row, b >> 1) + (b & 1) * 8, q[l].x, q[l].y);
                                asm volatile("st.shared.u8 [%0], %1;" ::"r"(sf_to + (b >> 2) * 512 + (row % 32) * 16 +
                                                                            row / 32 * 4 + (b & 3)),
                                             "r"(sf[l])
                                             : "memory");
                            }
                        }
                    }
                } else {
                    const int parts = DOWN ? 2 : 1;
                    for (int u0 = half * 128; u0 < t.n * parts * 8; u0 += 256) {  // pieces of 8 values: row u / 8, piece u % 8
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
                                w[l] = __ldg(reinterpret_cast<const uint4*>(from + k));
                            }
                        }
                        if (!free && !warp_wait_or_die(a, s, &s->empty[st], ph ^ 1)) return;
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
                if (!free && !warp_wait_or_die(a, s, &s->empty[st], ph ^ 1)) return;
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&s->full[st]));
            }
            if (++st == a.stages) st = 0, ph ^= 1;
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

// `sums`: down's [T][kRows] of this block; a thread has two rows of its own.
template <bool NVFP4, bool DOWN>
__device__ __forceinline__ void result_role(const LayerArgs& a, Shared* s, const Routing& r, const Work<DOWN>& work,
                                            float* sums) {
    constexpr int kPairs = NVFP4 ? 3 : DOWN ? 8 : 16;  // pairs of 16 columns
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tasks = work.tasks();
    const uint32_t lanes = uint32_t(warp * 32) << 16;
    for (int i = 0; i < tasks; i++) {
        const Task t = work.task(a, r, i);
        const int buf = i & 1;
        const float* alphas = DOWN ? a.f.alpha2 : a.f.alpha13;
        const float alpha = alphas ? __ldg(alphas + t.e) : 1.0f;
        if (!warp_wait_or_die(a, s, &s->acc_full[buf], i >> 1 & 1)) return;
        tc_fence_after();
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
                const float unscale = alpha * (NVFP4 ? pow2(-s->shift[i % kShifts][j0 + j]) : 1.0f);
                const float y0 = pair_sum<NVFP4, DOWN>(v0, j) * unscale, y1 = pair_sum<NVFP4, DOWN>(v1, j) * unscale;
                if (DOWN) {
                    float* to = sums + (p / a.f.K) * kRows + warp * 32 + lane;
                    const float f = __ldg(a.f.w + p);
                    to[0] = fmaf(f, y0, to[0]);
                    to[128] = fmaf(f, y1, to[128]);
                } else {
                    const int row = t.block * 128 + warp * 32 + lane, I = a.f.I;
                    const float h = row < I ? swiglu(y0, y1) : 0.0f;
                    if (NVFP4) {
                        if (row < I) h_values(a.f)[int64_t(p) * I + row] = h;
                        const float m = warp_max(fabsf(h));
                        if (lane == 0 && row < I) h_largest(a.f)[int64_t(p) * h_parts(I) + row / 32] = m;
                    } else if (row < I) {
                        uint16_t* to = static_cast<uint16_t*>(a.f.workspace) + int64_t(p) * 2 * I + row;
                        const uint32_t hi = pack_bf16x2(h, 0.0f) & 0xffffu;
                        to[0] = uint16_t(hi);
                        to[I] = uint16_t(pack_bf16x2(h - bf16_lo(hi), 0.0f));
                    }
                }
            }
        }
    }
}

template <bool NVFP4, bool DOWN>
__global__ void __launch_bounds__(kThreads, 1)
    few_tokens_kernel(const __grid_constant__ LayerArgs a, const __grid_constant__ CUtensorMap map) {
    using S = Shape<NVFP4, DOWN>;
    extern __shared__ uint8_t raw[];
    __shared__ Shared shared;
    Shared* s = &shared;
    uint8_t* base = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);  // slots on swizzle atoms
    const uint32_t slots = smem_addr(base);
    float* sums = reinterpret_cast<float*>(base + a.stages * S::kSlot);
    uint8_t* lists = base + a.stages * S::kSlot + (DOWN ? sizeof(float) * kRows * a.f.T : 0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == kMmaWarp) tmem_alloc(smem_addr(&s->tmem), 512);
    if (threadIdx.x == 0) {
        s->dead = 0;
        for (int i = 0; i < a.stages; i++) {
            mbar_init(smem_addr(&s->full[i]), 3);  // the loads' issuer and two converters
            mbar_init(smem_addr(&s->empty[i]), 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(smem_addr(&s->acc_full[i]), 1);
            mbar_init(smem_addr(&s->acc_empty[i]), 4);
        }
        mbar_init(smem_addr(&s->shifts_ready), 2 * min(kTurns, a.stages));
        mbar_fence_init();
    }
    if (DOWN && warp < 4)
        for (int i = threadIdx.x; i < kRows * a.f.T; i += 128) sums[i] = 0.0f;  // a thread's own two rows
    pdl_wait();
    const Routing r = route(a.f, lists, S::kGroup, !DOWN && blockIdx.x == 0);
    const cg::cluster_group cluster = cg::this_cluster();
    const int rank = DOWN ? int(cluster.block_rank()) : 0, ranks = DOWN ? int(cluster.num_blocks()) : 1;
    const Work<DOWN> work(a, r, rank, ranks);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    if (warp < 4)
        result_role<NVFP4, DOWN>(a, s, r, work, sums);
    else if (warp == kLoadWarp) {
        if (lane == 0) load_role<NVFP4, DOWN>(a, s, r, work, slots, &map);
    } else if (warp == kMmaWarp) {
        mma_role<NVFP4, DOWN>(a, s, r, work, slots);
    } else {
        convert_role<NVFP4, DOWN>(a, s, r, work, slots, warp - kConvertWarp);
    }
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
    if (DOWN) {
        cluster.sync();
        for (int i = rank * kThreads + int(threadIdx.x); i < kRows * a.f.T; i += ranks * kThreads) {
            const int row = work.block * 128 + i % kRows;
            float y = 0.0f;
            for (int b = 0; b < ranks; b++) y += cluster.map_shared_rank(sums, b)[i];
            if (row < a.f.H) a.f.out[int64_t(i / kRows) * a.f.H + row] = uint16_t(pack_bf16x2(y, 0.0f));
        }
        cluster.sync();  // no block's sums go before the others have read them
    }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
template <bool NVFP4, bool DOWN>
cudaError_t launch_half(const LaunchCtx& ctx, const FewTokens& f) {
    using S = Shape<NVFP4, DOWN>;
    constexpr size_t kMost = 226 * 1024;  // dynamic shared memory beside the static part
    const int rows = DOWN ? f.H : f.I, k = DOWN ? f.I : f.H, pairs = f.T * f.K;
    LayerArgs a{f, 0, 0, NVFP4 ? k / 2 : 2 * k, (rows + 127) / 128, k};
    a.chunks = (a.row_bytes + 127) / 128;
    const size_t fixed = 1024 + (DOWN ? sizeof(float) * kRows * f.T : 0) + routing_bytes(pairs, f.E) + sizeof(Shared);
    a.stages = int(std::min<size_t>(kMaxStages, (kMost - fixed) / S::kSlot));
    const size_t smem = fixed - sizeof(Shared) + size_t(a.stages) * S::kSlot;

    CUtensorMap map;
    const uint64_t dims[4] = {uint64_t(a.row_bytes), uint64_t(rows), DOWN ? 1u : 2u, uint64_t(f.E)};
    const uint32_t box[4] = {128, DOWN ? 256u : 128u, DOWN ? 1u : 2u, 1};
    if (!make_map(&map, DOWN ? f.w2 : f.w13, 4, dims, box)) return cudaErrorInvalidValue;
    auto kern = few_tokens_kernel<NVFP4, DOWN>;
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (err != cudaSuccess) return err;

    const int experts = std::min(pairs, f.E);
    if (!DOWN) {
        // one block for each SM; fewer where there are fewer tasks
        const int64_t tasks = int64_t(pairs) * a.blocks;
        return launch_pdl(ctx, kern, dim3(unsigned(std::min<int64_t>(tasks, ctx.num_sms))), dim3(kThreads), smem, a, map);
    }
    const int owners = (a.blocks + 1) / 2;
    int ranks = 1;  // as many as there are SMs and experts for
    while (ranks < 8 && owners * ranks * 2 <= ctx.num_sms && ranks * 2 <= experts) ranks *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(owners * ranks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = ctx.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(ranks);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a, map);
}

}  // namespace

size_t few_tokens_workspace(int64_t T, int K, int, int I, int) {
    return size_t(T) * K * (size_t(I) + h_parts(I)) * sizeof(float);
}

cudaError_t launch_few_tokens(const LaunchCtx& ctx, const FewTokens& f) {
    cudaError_t err = f.nvfp4 ? launch_half<true, false>(ctx, f) : launch_half<false, false>(ctx, f);
    if (err != cudaSuccess) return err;
    return f.nvfp4 ? launch_half<true, true>(ctx, f) : launch_half<false, true>(ctx, f);
}

}  // namespace moe
