// moe_layer.cu -- a whole MoE layer for a few tokens in two kernels.
//
//   gate_up:  h(p) = silu(alpha1 W1g x) * (alpha1 W1u x) for every pair p = (token, slot), e its expert
//   down:     out[t] = bf16(sum over t's pairs of topk_weight * alpha2 * W2 h(p))
//
// Bound by reading each routed expert's weights once from DRAM, so the work is split over weight rows and
// every byte goes straight from DRAM to the registers of the warp that multiplies it. Warp products
// (m16n8k16) have weight rows as M and an expert's tokens as N: with one to a few tokens an expert the tensor
// core is far from its rate whatever instruction feeds it, and operands in registers save the way
// through shared memory. The order of k inside a product is free as long as both operands agree, so a lane
// takes 16 contiguous bytes of a weight row (32 NVFP4 or 8 bf16 values) and the matching values of x.
//
// NVFP4 weights become fp16 products value(code) * value(scale): both factors and their product (6
// significant bits, at most 2688) are exact in fp16, one conversion and one multiplication for two weights
// (63 weights per clock and SM in a register-only loop, against 35 by way of bf16 and 38 that DRAM delivers).
// x and h are brought to fp16 range by a power of two: x (8 significant bits) exactly but for values
// below 2^-39 of the largest, h as the sum of two fp16 values (22 bits). With bf16 weights x stays bf16
// and h is the sum of two bf16 values (16 bits).
//
// Sums: fp32 inside a warp, then over the warps of a block in the order of their index. No atomics.
#include <algorithm>
#include <cstdint>

#include "expert_rows.cuh"
#include "experts_launch.h"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxPairs = 1024;  // MOE_LAYER_MAX_TOKENS * MOE_MAX_TOPK
constexpr int kUnit = 32;        // weight rows of a block: 8 neighbours in each 32-row group of a 128-row scale block,
                                 // whose scales are 16 contiguous bytes a lane
constexpr int kPart = 512;       // values of x or h that a warp stages for 8 columns at a time
constexpr int kWarpSmem = 32 * (kPart / 4 * 2 + 64);  // bytes a warp stages in (at most 32 columns), and sums through

// ---------------------------------------------------------------------------
// weight rows
// ---------------------------------------------------------------------------
template <bool NVFP4>
struct Format {
    static constexpr int kLane = NVFP4 ? 32 : 8;       // values of one 16-byte load
    static constexpr int kStep = 4 * kLane;            // values of k that a warp takes at a time
    static constexpr int kPad = NVFP4 ? 32 : 64;       // bytes between staged columns: no bank conflicts
};

// The rows r0 + lane/4 + 32j (j < 4) of one matrix [rows, k], as two m16 tiles (j = 0, 1 and j = 2, 3).
template <bool NVFP4>
struct RowsPtr {
    const uint8_t* w;   // first row of this lane, at this lane's k
    const uint8_t* sf;  // its scale line
    int64_t stride;     // bytes from row to row + 32
    int valid;          // bit j: the row exists
};

template <bool NVFP4>
__device__ __forceinline__ RowsPtr<NVFP4> rows_ptr(const void* w, const uint8_t* sf, int64_t matrix, int rows, int k,
                                                   int r0, int lane) {
    const int g = lane >> 2, q = lane & 3;
    const int64_t row_bytes = NVFP4 ? k / 2 : 2 * int64_t(k);
    RowsPtr<NVFP4> p;
    p.w = static_cast<const uint8_t*>(w) + (matrix * rows + r0 + g) * row_bytes + q * 16;
    p.stride = 32 * row_bytes;
    p.sf = NVFP4 ? sf + ((matrix * ((rows + 127) / 128) + r0 / 128) * (k / 64) + (q >> 1)) * 512 + (r0 % 32 + g) * 16
                 : nullptr;
    p.valid = 0;
    for (int j = 0; j < 4; j++) p.valid |= (r0 + g + 32 * j < rows) << j;
    return p;
}

template <bool NVFP4>
__device__ __forceinline__ void load_tile(const RowsPtr<NVFP4>& p, int tile, int step, bool k_ok, uint4* v) {
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const int j = tile * 2 + h;
        v[h] = make_uint4(0, 0, 0, 0);
        if (k_ok && (p.valid >> j & 1)) v[h] = ld_stream_v4(p.w + j * p.stride + int64_t(step) * 64);
    }
}

__device__ __forceinline__ void mma_16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1, bool f16) {
    if (f16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// Where a staged 16-byte piece (8 values) of a column lies: piece j of lane quarter q inside a step. NVFP4
// lanes read 4 pieces each; turning every other quarter's pieces keeps eight lanes off each other's banks.
template <bool NVFP4>
__device__ __forceinline__ uint32_t piece_at(int step_in_part, int q, int j) {
    return step_in_part * Format<NVFP4>::kStep * 2 + (NVFP4 ? q * 64 + (j ^ (q >> 1)) * 16 : q * 16);
}

// acc[mt][nt] += rows x columns over the warp's steps first, first + stride, .. (n of them). MT row tiles from
// MT/2 matrices, NT tiles of 8 columns that stage(i, n, smem) brings to shared memory for steps i .. i + n.
template <bool NVFP4, int MT, int NT, typename Stage>
__device__ __forceinline__ void multiply(float (&acc)[MT][NT][4], const RowsPtr<NVFP4>* rows, int k, int first,
                                         int stride, int n, uint8_t* smem, int cols, Stage stage) {
    using F = Format<NVFP4>;
    constexpr int kPartSteps = kPart / NT / F::kStep;
    constexpr int kColumn = kPart / NT * 2 + F::kPad;  // bytes
    const int lane = threadIdx.x & 31, q = lane & 3;
    const uint32_t base = smem_addr(smem);
    uint32_t column[NT];  // a column beyond the last reads the last one: its products are not used
#pragma unroll
    for (int nt = 0; nt < NT; nt++) column[nt] = base + min(nt * 8 + (lane >> 2), cols - 1) * kColumn;

    uint4 v[MT][2], sf[MT / 2];
    auto k_ok = [&](int i) { return i < n && (first + i * stride) * F::kStep + q * F::kLane < k; };
    auto load_sf = [&](int i, int m) {
        sf[m] = make_uint4(0, 0, 0, 0);
        if (NVFP4 && k_ok(i)) sf[m] = ld_stream_v4(rows[m].sf + int64_t(first + i * stride) * 1024);
    };
#pragma unroll
    for (int mt = 0; mt < MT; mt++) {
        load_tile<NVFP4>(rows[mt / 2], mt & 1, first, k_ok(0), v[mt]);
        if (mt % 2 == 0) load_sf(0, mt / 2);
    }
    for (int i = 0; i < n; i++) {
        const int at = i % kPartSteps;
        if (at == 0) {
            __syncwarp();
            stage(i, min(kPartSteps, n - i), smem);
            __syncwarp();
        }
        const bool more = k_ok(i + 1);
        auto fetch = [&](int nt, int j) {
            uint4 b;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                         : "r"(column[nt] + piece_at<NVFP4>(at, q, j)));
            return b;
        };
        constexpr int kPieces = NVFP4 ? 4 : 1;
        uint4 kept[kPieces];
        if (NT == 1)
#pragma unroll
            for (int j = 0; j < kPieces; j++) kept[j] = fetch(0, j);
#pragma unroll
        for (int mt = 0; mt < MT; mt++) {
            uint32_t s[2][2];  // [row g, g + 8][block of 16]
            if constexpr (NVFP4) {
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const uint16_t two = uint16_t(word(sf[mt / 2], (mt & 1) * 2 + h) >> (16 * (q & 1)));
                    uint32_t f;
                    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"(two));
                    s[h][0] = __byte_perm(f, f, 0x1010);
                    s[h][1] = __byte_perm(f, f, 0x3232);
                }
                if (mt % 2 == 1) load_sf(i + 1, mt / 2);
            }
#pragma unroll
            for (int j = 0; j < kPieces; j++) {
                uint32_t lo[4], hi[4];  // rows g and g + 8, 8 values
                if constexpr (NVFP4) {
                    decode8(word(v[mt][0], j), s[0][j / 2], lo);
                    decode8(word(v[mt][1], j), s[1][j / 2], hi);
                } else {
                    lo[0] = v[mt][0].x, lo[1] = v[mt][0].y, lo[2] = v[mt][0].z, lo[3] = v[mt][0].w;
                    hi[0] = v[mt][1].x, hi[1] = v[mt][1].y, hi[2] = v[mt][1].z, hi[3] = v[mt][1].w;
                }
                const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
                for (int nt = 0; nt < NT; nt++) {
                    const uint4 b = NT == 1 ? kept[j] : fetch(nt, j);
                    mma_16816(acc[mt][nt], a0, b.x, b.y, NVFP4);
                    mma_16816(acc[mt][nt], a1, b.z, b.w, NVFP4);
                }
            }
            load_tile<NVFP4>(rows[mt / 2], mt & 1, first + (i + 1) * stride, more, v[mt]);
        }
    }
}

// 2^e as fp32, e in [-126, 127]
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// The power of two that brings a largest magnitude amax to [2^14, 2^15); 1 for 0.
__device__ __forceinline__ int fp16_shift(float amax) {
    return amax == 0.0f ? 0 : 14 - max(int(__float_as_uint(amax) >> 23) - 127, -110);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFullMask, v, o));
    return v;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The pairs from `first` on that name expert e, in order, into list[0..); returns how many. One warp.
template <typename Id>
__device__ __forceinline__ int pairs_of(const Id* ids, int pairs, int first, int e, uint16_t* list, int lane) {
    int n = 0;
    for (int p0 = first; p0 < pairs; p0 += 32) {
        const int p = p0 + lane;
        const bool is = p < pairs && ids[p] == e;
        const unsigned m = __ballot_sync(kFullMask, is);
        if (is) list[n + __popc(m & ((1u << lane) - 1))] = uint16_t(p);
        n += __popc(m);
    }
    return n;
}

// Workspace: h as two 2-byte parts [pairs][2][I], then (NVFP4) its powers of two [pairs][units].
__host__ __device__ __forceinline__ int h_units(int I) { return (I + 127) / 128 * 4; }

// ---------------------------------------------------------------------------
// gate and up
// ---------------------------------------------------------------------------
// Columns c0 .. c0 + 8 NT of the block's expert: h of the block's 32 rows into the workspace.
template <bool NVFP4, int NT>
__device__ __forceinline__ void gate_up_columns(const FewTokens& a, int e, int r0, const uint16_t* list, int cols,
                                                uint8_t* smem) {
    using F = Format<NVFP4>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int steps = (a.H + F::kStep - 1) / F::kStep;
    const int mine = steps > warp ? (steps - warp + kWarps - 1) / kWarps : 0;
    uint8_t* own = smem + warp * kWarpSmem;
    RowsPtr<NVFP4> rows[2];
    for (int half = 0; half < 2; half++)
        rows[half] = rows_ptr<NVFP4>(a.w13, a.w13_sf, int64_t(e) * 2 + half, a.I, a.H, r0, lane);

    // this warp's part of every column, scaled to fp16 by its own largest magnitude (lane c: column c's)
    int shift = 0;
    if (NVFP4) {
        for (int c = 0; c < cols; c++) {
            const uint16_t* x = a.x + int64_t(list[c] / a.K) * a.H;
            float amax = 0.0f;
            for (int i = 0; i < mine; i++) {
                const int k = (warp + i * kWarps) * F::kStep + lane * 4;
                if (k < a.H) {
                    const uint2 w = __ldg(reinterpret_cast<const uint2*>(x + k));
                    amax = fmaxf(amax, fmaxf(fmaxf(fabsf(bf16_lo(w.x)), fabsf(bf16_hi(w.x))),
                                             fmaxf(fabsf(bf16_lo(w.y)), fabsf(bf16_hi(w.y)))));
                }
            }
            const int sh = fp16_shift(warp_max(amax));
            if (lane == c) shift = sh;
        }
    }
    auto stage = [&](int i, int n, uint8_t* to) {
        constexpr int kColumn = kPart / NT * 2 + F::kPad;
        const int pieces = n * F::kStep / 8;
        for (int c = 0; c < cols; c++) {
            const uint16_t* x = a.x + int64_t(list[c] / a.K) * a.H;
            const float scale = pow2(__shfl_sync(kFullMask, shift, c));
            for (int p = lane; p < pieces; p += 32) {
                const int st = p / (F::kStep / 8), in = p % (F::kStep / 8);
                const int k = (warp + (i + st) * kWarps) * F::kStep + in * 8;
                uint4 w = make_uint4(0, 0, 0, 0);
                if (k < a.H) w = __ldg(reinterpret_cast<const uint4*>(x + k));
                if (NVFP4) {
                    float f[8];
                    unpack8(w, f);
                    for (int j = 0; j < 8; j++) f[j] *= scale;
                    w = make_uint4(pack_f16x2(f[0], f[1]), pack_f16x2(f[2], f[3]), pack_f16x2(f[4], f[5]),
                                   pack_f16x2(f[6], f[7]));
                }
                *reinterpret_cast<uint4*>(to + c * kColumn + (NVFP4 ? piece_at<true>(st, in >> 2, in & 3)
                                                                    : piece_at<false>(st, in, 0))) = w;
            }
        }
    };
    float acc[4][NT][4] = {};
    multiply<NVFP4, 4, NT>(acc, rows, a.H, warp, kWarps, mine, own, cols, stage);

    // sums of the warps: [warp][gate 32 rows, up 32 rows][8 NT columns]
    __syncwarp();
    float* sums = reinterpret_cast<float*>(own);
    const int g = lane >> 2, q = lane & 3;
#pragma unroll
    for (int mt = 0; mt < 4; mt++)
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int c = nt * 8 + q * 2 + (j & 1), row = mt * 16 + (j >> 1) * 8 + g;
                const float inv = NVFP4 ? pow2(-__shfl_sync(kFullMask, shift, c)) : 1.0f;
                sums[row * 8 * NT + c] = acc[mt][nt][j] * inv;
            }
    __syncthreads();
    const float alpha = a.alpha13 ? __ldg(a.alpha13 + e) : 1.0f;
    const int row = r0 + lane % 8 + 32 * (lane / 8);  // the order of sums' rows
    for (int c = warp; c < cols; c += kWarps) {
        float gate = 0.0f, up = 0.0f;
        for (int w = 0; w < kWarps; w++) {
            const float* sw = reinterpret_cast<const float*>(smem + w * kWarpSmem);
            gate += sw[lane * 8 * NT + c];
            up += sw[(32 + lane) * 8 * NT + c];
        }
        const float h = row < a.I ? swiglu(alpha * gate, alpha * up) : 0.0f;
        const int64_t p = list[c];
        uint16_t* to = static_cast<uint16_t*>(a.workspace) + p * 2 * a.I;
        uint32_t hi, lo;
        if (NVFP4) {
            const float amax = warp_max(fabsf(h));
            const int sh = fp16_shift(amax);
            const float v = h * pow2(sh);
            hi = pack_f16x2(v, 0.0f) & 0xffffu;
            lo = pack_f16x2(v - __half2float(__ushort_as_half(uint16_t(hi))), 0.0f);
            if (lane == 0) {
                float* inv = reinterpret_cast<float*>(static_cast<uint16_t*>(a.workspace) + int64_t(a.T) * a.K * 2 * a.I);
                inv[p * h_units(a.I) + r0 / 128 * 4 + r0 % 32 / 8] = amax > 0.0f ? pow2(-sh) : 0.0f;
            }
        } else {
            hi = pack_bf16x2(h, 0.0f) & 0xffffu;
            lo = pack_bf16x2(h - bf16_lo(hi), 0.0f);
        }
        if (row < a.I) {
            to[row] = uint16_t(hi);
            to[a.I + row] = uint16_t(lo);
        }
    }
    __syncthreads();
}

// Block (unit, pair): the pair is the first of its expert, or there is nothing to do.
template <bool NVFP4, int MAXNT>
__global__ void __launch_bounds__(kThreads, 2) few_tokens_gate_up_kernel(FewTokens a) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ uint16_t list[kMaxPairs];
    __shared__ int count;
    pdl_wait();
    const int pair = blockIdx.y, pairs = a.T * a.K;
    const int e = __ldg(a.ids + pair);
    if (e < 0 || e >= a.E) {
        if (e != -1 && blockIdx.x == 0 && threadIdx.x == 0) set_status(a.status, MOE_ERR_BAD_EXPERT_ID);
        return;
    }
    int earlier = 0;
    for (int p = threadIdx.x; p < pair; p += kThreads) earlier |= __ldg(a.ids + p) == e;
    if (__syncthreads_or(earlier)) return;
    if (threadIdx.x < 32) {
        const int n = pairs_of(a.ids, pairs, pair, e, list, threadIdx.x);
        if (threadIdx.x == 0) count = n;
    }
    __syncthreads();
    const int n = count;
    const int r0 = int(blockIdx.x) / 4 * 128 + int(blockIdx.x) % 4 * 8;
    if (r0 >= a.I) return;
    if (MAXNT == 1 || n <= 8) {
        for (int c = 0; c < n; c += 8) gate_up_columns<NVFP4, 1>(a, e, r0, list + c, min(8, n - c), smem);
    } else if (MAXNT == 2 || n <= 16) {
        for (int c = 0; c < n; c += 16)
            gate_up_columns<NVFP4, MAXNT == 1 ? 1 : 2>(a, e, r0, list + c, min(16, n - c), smem);
    } else {
        for (int c = 0; c < n; c += 32) gate_up_columns<NVFP4, MAXNT>(a, e, r0, list + c, min(32, n - c), smem);
    }
}

// ---------------------------------------------------------------------------
// down
// ---------------------------------------------------------------------------
// Pairs list[0 .. n) of expert e (at most 4 NT: columns are the two parts of each h): the warp's steps
// added, weighted, to its sums [32 rows][T].
template <bool NVFP4, int NT>
__device__ __forceinline__ void down_columns(const FewTokens& a, int e, int r0, const uint16_t* list, int n, int first,
                                             int steps, uint8_t* own, float* sums) {
    using F = Format<NVFP4>;
    const int lane = threadIdx.x & 31;
    const RowsPtr<NVFP4> rows = rows_ptr<NVFP4>(a.w2, a.w2_sf, e, a.H, a.I, r0, lane);
    const uint16_t* hp = static_cast<const uint16_t*>(a.workspace);
    const float* inv = reinterpret_cast<const float*>(hp + int64_t(a.T) * a.K * 2 * a.I);
    const int units = h_units(a.I);

    float largest = 1.0f;  // NVFP4: lane c's is the largest power of two of pair c, to which all are brought
    if (NVFP4) {
        for (int c = 0; c < n; c++) {
            float m = 0.0f;
            for (int u = lane; u < units; u += 32)
                if (u / 4 * 128 + u % 4 * 8 < a.I) m = fmaxf(m, __ldg(inv + int64_t(list[c]) * units + u));
            m = warp_max(m);
            if (lane == c && m > 0.0f) largest = m;
        }
    }
    auto stage = [&](int i, int count, uint8_t* to) {
        constexpr int kColumn = kPart / NT * 2 + F::kPad;
        const int pieces = count * F::kStep / 8;
        for (int c = 0; c < n; c++) {
            const float unscale = 1.0f / __shfl_sync(kFullMask, largest, c);  // of a power of two: exact
            const uint16_t* h = hp + int64_t(list[c]) * 2 * a.I;
            // columns of a tile of 8: four pairs' first parts, then their second parts
            uint8_t* column = to + ((c & 3) + c / 4 * 8) * kColumn;
            for (int p = lane; p < pieces; p += 32) {
                const int st = p / (F::kStep / 8), in = p % (F::kStep / 8);
                const int k = (first + i + st) * F::kStep + in * 8;
                uint4 w[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
                if (k < a.I) {
                    w[0] = __ldg(reinterpret_cast<const uint4*>(h + k));
                    w[1] = __ldg(reinterpret_cast<const uint4*>(h + a.I + k));
                    if (NVFP4) {
                        const float f = __ldg(inv + int64_t(list[c]) * units + k / 128 * 4 + k % 32 / 8) * unscale;
                        const uint32_t f2 = pack_f16x2(f, f);
                        for (int j = 0; j < 2; j++)
                            asm("mul.rn.f16x2 %0, %0, %4;\n\tmul.rn.f16x2 %1, %1, %4;\n\t"
                                "mul.rn.f16x2 %2, %2, %4;\n\tmul.rn.f16x2 %3, %3, %4;"
                                : "+r"(w[j].x), "+r"(w[j].y), "+r"(w[j].z), "+r"(w[j].w)
                                : "r"(f2));
                    }
                }
                const uint32_t at = NVFP4 ? piece_at<true>(st, in >> 2, in & 3) : piece_at<false>(st, in, 0);
                *reinterpret_cast<uint4*>(column + at) = w[0];
                *reinterpret_cast<uint4*>(column + 4 * kColumn + at) = w[1];
            }
        }
    };
    float acc[2][NT][4] = {};
    multiply<NVFP4, 2, NT>(acc, &rows, a.I, first, 1, steps, own, 8 * NT, stage);

    const float alpha = a.alpha2 ? __ldg(a.alpha2 + e) : 1.0f;
    const int g = lane >> 2, q = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
        float y[2][4];
#pragma unroll
        for (int mt = 0; mt < 2; mt++)
#pragma unroll
            for (int j = 0; j < 4; j++)  // first part (lanes q < 2) + second part
                y[mt][j] = acc[mt][nt][j] + __shfl_xor_sync(kFullMask, acc[mt][nt][j], 2);
#pragma unroll
        for (int turn = 0; turn < 2; turn++) {  // one lane after the other: an expert may have a token twice
#pragma unroll
            for (int j1 = 0; j1 < 2; j1++) {
                const int c = nt * 4 + turn * 2 + j1;
                const float big = __shfl_sync(kFullMask, largest, c & 31);
                if (q == turn && c < n) {
                    const int p = list[c];
                    const float f = __ldg(a.w + p) * alpha * big;
                    float* to = sums + p / a.K;
#pragma unroll
                    for (int mt = 0; mt < 2; mt++)
#pragma unroll
                        for (int j0 = 0; j0 < 2; j0++) {
                            float* at = to + (mt * 16 + j0 * 8 + g) * a.T;
                            *at = fmaf(f, y[mt][j0 * 2 + j1], *at);
                        }
                }
            }
            __syncwarp();
        }
    }
}

template <bool NVFP4, int MAXNT>
__global__ void __launch_bounds__(kThreads, 2) few_tokens_down_kernel(FewTokens a) {
    // every warp's staging and its sums [32][T]; the experts' first pairs; the pairs' ids, the first pairs in
    // order, every warp's list of pairs
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int n_first;
    using F = Format<NVFP4>;
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int pairs = a.T * a.K;
    int* owner = reinterpret_cast<int*>(smem + kWarps * (kWarpSmem + kUnit * a.T * sizeof(float)));
    int16_t* ids = reinterpret_cast<int16_t*>(owner + a.E);
    uint16_t* firsts = reinterpret_cast<uint16_t*>(ids + pairs);
    uint16_t* list = firsts + pairs + warp * pairs;
    const int r0 = int(blockIdx.x) / 4 * 128 + int(blockIdx.x) % 4 * 8;
    if (r0 >= a.H) return;
    float* sums = reinterpret_cast<float*>(smem + kWarps * kWarpSmem) + warp * kUnit * a.T;
    for (int i = lane; i < kUnit * a.T; i += 32) sums[i] = 0.0f;
    for (int e = threadIdx.x; e < a.E; e += kThreads) owner[e] = kMaxPairs;
    __syncthreads();
    for (int p = threadIdx.x; p < pairs; p += kThreads) {
        const int e = __ldg(a.ids + p);
        ids[p] = int16_t(e >= 0 && e < a.E ? e : -1);
        if (ids[p] >= 0) atomicMin(&owner[e], p);
    }
    __syncthreads();
    if (warp == 0) {  // the first pair of every routed expert, in order
        int n = 0;
        for (int p0 = 0; p0 < pairs; p0 += 32) {
            const int p = p0 + lane;
            const bool is = p < pairs && ids[p] >= 0 && owner[ids[p]] == p;
            const unsigned m = __ballot_sync(kFullMask, is);
            if (is) firsts[n + __popc(m & ((1u << lane) - 1))] = uint16_t(p);
            n += __popc(m);
        }
        if (lane == 0) n_first = n;
    }
    __syncthreads();

    // items: an expert's steps, cut in parts while there are few experts
    const int steps = (a.I + F::kStep - 1) / F::kStep;
    const int cut = min(steps, max(1, (2 * kWarps + n_first - 1) / max(1, n_first)));
    const int per = (steps + cut - 1) / cut;
    uint8_t* own = smem + warp * kWarpSmem;
    for (int item = warp; item < n_first * cut; item += kWarps) {
        const int pair = firsts[item / cut], first = item % cut * per;
        const int n_steps = min(per, steps - first);
        if (n_steps <= 0) continue;
        const int e = ids[pair];
        __syncwarp();
        const int n = pairs_of(ids, pairs, pair, e, list, lane);
        __syncwarp();
        for (int c = 0; c < n;) {
            const int left = n - c;
            if (MAXNT == 1 || left <= 4) {
                down_columns<NVFP4, 1>(a, e, r0, list + c, min(4, left), first, n_steps, own, sums);
                c += 4;
            } else if (MAXNT == 2 || left <= 8) {
                down_columns<NVFP4, MAXNT == 1 ? 1 : 2>(a, e, r0, list + c, min(8, left), first, n_steps, own, sums);
                c += 8;
            } else {
                down_columns<NVFP4, MAXNT>(a, e, r0, list + c, min(16, left), first, n_steps, own, sums);
                c += 16;
            }
        }
    }
    __syncthreads();
    const float* all = reinterpret_cast<const float*>(smem + kWarps * kWarpSmem);
    for (int i = threadIdx.x; i < kUnit * a.T; i += kThreads) {
        const int r = i % kUnit, t = i / kUnit;
        const int row = r0 + r % 8 + 32 * (r / 8);
        float y = 0.0f;
        for (int w = 0; w < kWarps; w++) y += all[(w * kUnit + r) * a.T + t];
        if (row < a.H) a.out[int64_t(t) * a.H + row] = uint16_t(pack_bf16x2(y, 0.0f));
    }
}

template <bool NVFP4, int MAXNT>
cudaError_t launch(const LaunchCtx& ctx, const FewTokens& a) {
    const size_t s1 = size_t(kWarps) * kWarpSmem, s2 = s1 + size_t(kWarps) * kUnit * a.T * sizeof(float) +
                                                              a.E * sizeof(int) + (kWarps + 2) * sizeof(int16_t) * a.T * a.K;
    auto k1 = few_tokens_gate_up_kernel<NVFP4, MAXNT>;
    auto k2 = few_tokens_down_kernel<NVFP4, MAXNT>;
    cudaError_t err = cudaFuncSetAttribute(k1, cudaFuncAttributeMaxDynamicSharedMemorySize, int(s1));
    if (err == cudaSuccess) err = cudaFuncSetAttribute(k2, cudaFuncAttributeMaxDynamicSharedMemorySize, int(s2));
    if (err == cudaSuccess)
        err = launch_pdl(ctx, k1, dim3(unsigned(h_units(a.I)), unsigned(a.T * a.K)), dim3(kThreads), s1, a);
    if (err == cudaSuccess) err = launch_pdl(ctx, k2, dim3(unsigned(h_units(a.H))), dim3(kThreads), s2, a);
    return err;
}

}  // namespace

size_t few_tokens_workspace(int64_t T, int K, int, int I, int) {
    return size_t(T) * K * (size_t(2) * I * sizeof(uint16_t) + size_t(h_units(I)) * sizeof(float));
}

cudaError_t launch_few_tokens(const LaunchCtx& ctx, const FewTokens& a) {
    // with 8 tokens an expert has at most 8 columns (unless a token names it twice): fewer registers
    if (a.T <= 8) return a.nvfp4 ? launch<true, 1>(ctx, a) : launch<false, 1>(ctx, a);
    return a.nvfp4 ? launch<true, 2>(ctx, a) : launch<false, 4>(ctx, a);
}

}  // namespace moe
