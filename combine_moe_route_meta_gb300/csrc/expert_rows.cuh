// expert_rows.cuh -- device helpers shared by the expert operators.
#pragma once

#include "block_launch.h"
#include "dispatch_slice.cuh"
#include "experts_launch.h"
#include "moe_device.cuh"

namespace moe {

// A block of 16 values as NVFP4: its codes, and the scale, in the binary32 steps of the dispatch: sf = e4m3((amax / 6) * g),
// r = g / value(sf), q = e2m1(x * r); all codes 0 where value(sf) is 0. A product with the rounded 1/6 would give blocks on a
// boundary another scale than the dispatch gives them (and 32 experts' weights 1 % less time).
__device__ __forceinline__ uint2 quantise_block(const float (&f)[16], float g, uint32_t* sf) {
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 16; j++) amax = fmaxf(amax, fabsf(f[j]));
    *sf = e4m3x2(__fmul_rn(__fdiv_rn(amax, 6.0f), g), 0.0f) & 0xffu;
    const float s = e4m3_value(*sf);
    if (s == 0.0f) return make_uint2(0, 0);
    const float r = __fdiv_rn(g, s);
    uint32_t b[8];
#pragma unroll
    for (int p = 0; p < 8; p++) b[p] = e2m1x2(__fmul_rn(f[2 * p], r), __fmul_rn(f[2 * p + 1], r));
    return make_uint2(b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24, b[4] | b[5] << 8 | b[6] << 16 | b[7] << 24);
}

// 32 bytes to a 32-byte aligned address
__device__ __forceinline__ void st_v8(void* p, const uint32_t* w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// The rows [base, base + count) of expert e, cut to the layout's capacity.
struct RowSpan {
    int64_t base;
    int count;
};
__device__ __forceinline__ RowSpan expert_rows(const RowLayout& a, int e) {
    const int64_t base = a.M > 0 ? int64_t(e) * a.M : __ldg(a.seg + e);
    int64_t count = __ldg(a.count + e);
    if (count < 0 || base < 0) {
        set_status(a.status, MOE_ERR_INVALID_ARG);
        return RowSpan{0, 0};
    }
    const int64_t most = a.M > 0 ? a.M : max(a.rows - base, int64_t(0));
    if (count > most) {
        set_status(a.status, MOE_ERR_CAPACITY);
        count = most;
    }
    return RowSpan{base, int(count)};
}
__device__ __forceinline__ RowSpan expert_rows(const ExpertGemm& a, int e) {
    return expert_rows(RowLayout{a.E, a.M, a.rows, a.seg, a.count, a.status}, e);
}

// Byte offset of the scale of block c of row r of an activation matrix with C blocks a row.
__device__ __forceinline__ int64_t act_sf_index(int layout, int64_t r, int c, int C) {
    return layout == MOE_SCALES_SWIZZLED_128X4 ? swizzled_128x4_index(r, c, C) : r * C + c;
}

// up * gate / (1 + exp(-gate)) to 2^-20, with exp(-|gate|) = e c: the quotient is gate / (1 + e c), times e c below 0, so
// that nothing overflows and no gate's value is lost that a large `up` could make count. e = 2^t, t = -|gate| log2(e), and
// c = 1 + d ln 2 puts back t's rounding error d (grown with |gate|) to first order. 2^t (subnormal values too) and the
// reciprocal are the approximate instructions. Beyond 110 e is 0 in binary32.
__device__ __forceinline__ float swiglu(float gate, float up) {
    constexpr float kLog2e = 1.44269504f, kRest = 1.92596299e-8f, kLn2 = 0.693147181f;  // log2(e) = kLog2e + kRest
    float g;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(g) : "f"(gate), "f"(-110.0f));
    const float a = fminf(fabsf(g), 110.0f);
    const float t = -a * kLog2e;
    const float c = fmaf(fmaf(-a, kLog2e, -t) - a * kRest, kLn2, 1.0f);
    float e, r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(t));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(e, c, 1.0f)));
    // e by itself: a subnormal e is not rounded twice, nor its small product with gate
    return g < 0.0f ? (up * e) * (g * r * c) : up * (g * r);
}

// p = 1 / (1 + exp(-g)) and q = 1 - p, each to 2^-20 and the step of a subnormal exp(-|g|): by e = exp(-|g|), made as in
// swiglu(), one is 1 / (1 + e) and the other e / (1 + e), so neither is a difference.
__device__ __forceinline__ void sigmoids(float g, float* p, float* q) {
    constexpr float kLog2e = 1.44269504f, kRest = 1.92596299e-8f, kLn2 = 0.693147181f;
    const float a = fminf(fabsf(g), 110.0f);
    const float t = -a * kLog2e;
    const float c = fmaf(fmaf(-a, kLog2e, -t) - a * kRest, kLn2, 1.0f);
    float e, r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(t));
    e *= c;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e + 1.0f));
    *p = g < 0.0f ? e * r : r;
    *q = g < 0.0f ? r : e * r;
}
// The gradient of h = up * silu(gate) with respect to gate and up, times dh. In this order no factor overflows, or becomes
// 0 times infinity, where the result does not: below 0 gate counts after p has made it small.
__device__ __forceinline__ void dswiglu(float gate, float up, float dh, float* dgate, float* dup) {
    float p, q;
    sigmoids(gate, &p, &q);
    *dgate = dh * ((up * p) * fmaf(gate, q, 1.0f));
    *dup = dh * (gate * p);
}

}  // namespace moe
