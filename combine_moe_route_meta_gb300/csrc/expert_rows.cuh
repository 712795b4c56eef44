// expert_rows.cuh -- device helpers shared by the expert operators.
#pragma once

#include "dispatch_slice.cuh"
#include "experts_launch.h"
#include "moe_device.cuh"

namespace moe {

// value of an e2m1 code (its low three bits: 0, 0.5, 1, 1.5, 2, 3, 4, 6; bit 3 the sign)
__device__ __forceinline__ float e2m1_value(uint32_t code) {
    const uint32_t m = code & 7u;
    const float v = m < 2 ? 0.5f * float(m) : __uint_as_float(((126u + (m >> 1)) << 23) | ((m & 1u) << 22));
    return (code & 8u) ? -v : v;
}

// The rows [base, base + count) of expert e, cut to the layout's capacity.
struct RowSpan {
    int64_t base;
    int count;
};
__device__ __forceinline__ RowSpan expert_rows(const ExpertGemm& a, int e) {
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

// Byte offset of the scale of block c of row r of an activation matrix with C blocks a row.
__device__ __forceinline__ int64_t act_sf_index(int layout, int64_t r, int c, int C) {
    return layout == MOE_SCALES_SWIZZLED_128X4 ? swizzled_128x4_index(r, c, C) : r * C + c;
}

// h = up * silu(gate)
__device__ __forceinline__ float swiglu(float gate, float up) { return up * (gate / (1.0f + expf(-gate))); }

}  // namespace moe
