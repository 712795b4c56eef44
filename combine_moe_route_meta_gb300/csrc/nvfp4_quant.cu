// nvfp4_quant.cu -- bf16 rows to NVFP4 codes and block scales, and back.
//
//   quantise:    sf = e4m3((amax16 / 6) * g),  q = e2m1(x * (g / sf))   (dispatch_slice.cuh's arithmetic)
//   dequantise:  out = bf16((value(q) * value(sf)) / g)
//
// One thread per block of 16 elements: it reads (or writes) 32 contiguous bytes of a bf16 row and
// writes (or reads) 8 bytes of codes and one scale byte, so a block's amax needs no shuffle.
// Bound by DRAM: 2.5625 bytes per element.
#include <algorithm>
#include <cstdint>

#include "expert_rows.cuh"
#include "experts_launch.h"

namespace moe {
namespace {

constexpr int kQuantThreads = 256;

struct QuantArgs {
    const uint16_t* x;
    uint16_t* out;
    uint8_t* codes;
    uint8_t* sf;
    const float* gs;
    int64_t G, R, Rp;  // groups, rows, rows with the padding of the tiles
    int C;             // blocks per row
};

template <bool SWIZZLED>
__device__ __forceinline__ int64_t sf_index(const QuantArgs& a, int64_t g, int64_t r, int c) {
    if (SWIZZLED) return g * a.Rp * a.C + swizzled_128x4_index(r, c, a.C);
    return (g * a.R + r) * a.C + c;
}

template <bool SWIZZLED>
__global__ void __launch_bounds__(kQuantThreads) quantize_kernel(QuantArgs a) {
    pdl_wait();
    const int64_t n = a.G * a.Rp * a.C;
    for (int64_t i = int64_t(blockIdx.x) * kQuantThreads + threadIdx.x; i < n; i += int64_t(gridDim.x) * kQuantThreads) {
        const int c = int(i % a.C);
        const int64_t gr = i / a.C, g = gr / a.Rp, r = gr - g * a.Rp;
        uint32_t sf = 0;
        if (r < a.R) {
            const int64_t at = (g * a.R + r) * a.C + c;
            const LaneCodes q = quantise16<MOE_QUANT_NVFP4_B16>(load_slice(a.x + at * 16), __ldg(a.gs + g));
            st_v2(a.codes + at * 8, make_uint2(q.q.x, q.q.y));
            sf = q.scale;
        }
        a.sf[sf_index<SWIZZLED>(a, g, r, c)] = uint8_t(sf);
    }
}

template <bool SWIZZLED>
__global__ void __launch_bounds__(kQuantThreads) dequantize_kernel(QuantArgs a) {
    pdl_wait();
    const int64_t n = a.G * a.R * a.C;
    for (int64_t i = int64_t(blockIdx.x) * kQuantThreads + threadIdx.x; i < n; i += int64_t(gridDim.x) * kQuantThreads) {
        const int c = int(i % a.C);
        const int64_t gr = i / a.C, g = gr / a.R, r = gr - g * a.R;
        const uint2 q = *reinterpret_cast<const uint2*>(a.codes + i * 8);
        const float sf = e4m3_value(a.sf[sf_index<SWIZZLED>(a, g, r, c)]);
        const float gs = __ldg(a.gs + g);
        uint32_t w[8];
#pragma unroll
        for (int p = 0; p < 8; p++) {
            const uint32_t b = ((p < 4 ? q.x : q.y) >> (8 * (p & 3))) & 0xffu;
            w[p] = pack_bf16x2(__fdiv_rn(e2m1_value(b) * sf, gs), __fdiv_rn(e2m1_value(b >> 4) * sf, gs));
        }
        st_v4(a.out + i * 16, make_uint4(w[0], w[1], w[2], w[3]));
        st_v4(a.out + i * 16 + 8, make_uint4(w[4], w[5], w[6], w[7]));
    }
}

unsigned quant_grid(const LaunchCtx& ctx, int64_t blocks) {
    const int64_t need = (blocks + kQuantThreads - 1) / kQuantThreads;
    return unsigned(std::max<int64_t>(1, std::min<int64_t>(need, int64_t(ctx.num_sms) * 8)));
}

}  // namespace

cudaError_t launch_quantize_nvfp4(const LaunchCtx& ctx, const uint16_t* x, int64_t G, int64_t R, int H,
                                  const float* gs, int scale_layout, uint8_t* codes, uint8_t* scales) {
    const bool sw = scale_layout == MOE_SCALES_SWIZZLED_128X4;
    QuantArgs a{x, nullptr, codes, scales, gs, G, R, sw ? (R + 127) / 128 * 128 : R, H / 16};
    const unsigned grid = quant_grid(ctx, a.G * a.Rp * a.C);
    return launch_pdl(ctx, sw ? quantize_kernel<true> : quantize_kernel<false>, dim3(grid), dim3(kQuantThreads), 0, a);
}

cudaError_t launch_dequantize_nvfp4(const LaunchCtx& ctx, const uint8_t* codes, const uint8_t* scales, int64_t G,
                                    int64_t R, int H, const float* gs, int scale_layout, uint16_t* out) {
    const bool sw = scale_layout == MOE_SCALES_SWIZZLED_128X4;
    QuantArgs a{nullptr, out, const_cast<uint8_t*>(codes), const_cast<uint8_t*>(scales), gs, G, R,
                sw ? (R + 127) / 128 * 128 : R, H / 16};
    const unsigned grid = quant_grid(ctx, a.G * a.R * a.C);
    return launch_pdl(ctx, sw ? dequantize_kernel<true> : dequantize_kernel<false>, dim3(grid), dim3(kQuantThreads), 0,
                      a);
}

}  // namespace moe
