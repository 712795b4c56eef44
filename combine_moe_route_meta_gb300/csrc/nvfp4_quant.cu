// nvfp4_quant.cu -- bf16 rows to NVFP4 codes and block scales, and back.
//
//   quantise:    sf = e4m3((amax16 / 6) * g),  q = e2m1(x * (g / sf))   (quantise_block)
//   dequantise:  out = bf16((value(q) * value(sf)) / g)
//
// A thread takes one block of 16 elements at a time: 32 contiguous bytes of a bf16 row, 8 bytes of codes and
// one scale byte, so a block's amax needs no shuffle; four neighbouring threads join their scales to a word.
// A thread block takes kQuantRows rows x 64 CC columns, whose scales lie next to each other in the 512-byte tiles, and
// issues all its loads before it computes. Bound by DRAM: 2.5625 bytes per element. 32 experts' weights of 2048 x 7168
// quantised and read back, 2.4 GB, take 364 us (6.6 TB/s, 97 % of the copy bandwidth); 3 x 1001 x 4160 values 14.2 us
// and 128 x 7168 values 3.6 us for the two launches, whose starts and ends these are.
#include <algorithm>
#include <cstdint>

#include "expert_rows.cuh"
#include "experts_launch.h"

namespace moe {
namespace {

constexpr int kQuantThreads = 256;
// Rows of a thread block. Smaller ones leave more blocks to an SM: 32 experts' weights (0.94 GB) quantised in
// 218 us with 128, 193 us with 64 (before a block's scale took a division).
constexpr int kQuantRows = 64;

struct QuantArgs {
    const uint16_t* x;
    uint16_t* out;
    uint8_t* codes;
    uint8_t* sf;
    const float* gs;
    int64_t tiles;        // of kQuantRows rows x 64 CC columns, over all groups
    int R, C;             // rows and blocks per row of a group
    int row_tiles, chunks;  // tiles of a group: row_tiles x chunks
    bool wide;            // bf16 rows are 32-byte aligned
    bool sf_words;        // four neighbouring blocks' scales are a word (always so in the tiles)
};

// Where a thread's blocks lie: column block c of rows r, r + step, .. of group g.
struct QuantPlace {
    int g, r, c;
};

template <int CC>
__device__ __forceinline__ QuantPlace quant_place(const QuantArgs& a, int64_t tile) {
    const int chunk = int(tile % a.chunks);
    const int64_t gr = tile / a.chunks;
    const int g = int(gr / a.row_tiles);
    return QuantPlace{g, int(gr - int64_t(g) * a.row_tiles) * kQuantRows + int(threadIdx.x) / (4 * CC),
                      chunk * 4 * CC + int(threadIdx.x) % (4 * CC)};
}

// Scale of block (r, c) of group g; with the tiles, a group's matrix has its rows padded to whole tiles.
template <bool SWIZZLED>
__device__ __forceinline__ int64_t sf_index(const QuantArgs& a, const QuantPlace& p, int r) {
    if (SWIZZLED) return int64_t(p.g) * ((a.R + 127) / 128 * 128) * a.C + swizzled_128x4_index(r, p.c, a.C);
    return (int64_t(p.g) * a.R + r) * a.C + p.c;
}

__device__ __forceinline__ LaneSlice load_block(const uint16_t* p, bool wide) {
    if (!wide) return load_slice(p);
    LaneSlice s;
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(s.v0.x), "=r"(s.v0.y), "=r"(s.v0.z), "=r"(s.v0.w), "=r"(s.v1.x), "=r"(s.v1.y), "=r"(s.v1.z),
                   "=r"(s.v1.w)
                 : "l"(p));
    return s;
}

template <int CC, bool SWIZZLED>
__global__ void __launch_bounds__(kQuantThreads) quantize_kernel(QuantArgs a) {
    pdl_wait();
    constexpr int kStep = kQuantThreads / (4 * CC), kTurns = kQuantRows / kStep;
    for (int64_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
        const QuantPlace p = quant_place<CC>(a, tile);
        const int64_t at = (int64_t(p.g) * a.R + p.r) * a.C + p.c;  // block of the first row
        LaneSlice v[kTurns];
#pragma unroll
        for (int i = 0; i < kTurns; i++) {
            v[i].v0 = v[i].v1 = make_uint4(0, 0, 0, 0);
            if (p.r + i * kStep < a.R && p.c < a.C) v[i] = load_block(a.x + (at + int64_t(i) * kStep * a.C) * 16, a.wide);
        }
        const float gs = __ldg(a.gs + p.g);
#pragma unroll
        for (int i = 0; i < kTurns; i++) {
            const int r = p.r + i * kStep;
            const bool live = r < a.R && p.c < a.C;
            float f[16];
            unpack8(v[i].v0, f);
            unpack8(v[i].v1, f + 8);
            uint32_t sf;
            const uint2 q = quantise_block(f, gs, &sf);
            if (live) st_v2(a.codes + (at + int64_t(i) * kStep * a.C) * 8, q);
            if (SWIZZLED || a.sf_words) {  // zero in the padding rows of a tile
                uint32_t w = live ? sf << (8 * (threadIdx.x & 3)) : 0u;
                w |= __shfl_xor_sync(kFullMask, w, 1);
                w |= __shfl_xor_sync(kFullMask, w, 2);
                if ((threadIdx.x & 3) == 0 && p.c < a.C && (SWIZZLED || r < a.R))
                    *reinterpret_cast<uint32_t*>(a.sf + sf_index<SWIZZLED>(a, p, r)) = w;
            } else if (live) {
                a.sf[sf_index<SWIZZLED>(a, p, r)] = uint8_t(sf);
            }
        }
    }
}

// The eight magnitudes of a block as bf16 bytes, to be picked by code: lo/hi[i] hold those of codes 4i .. 4i + 3.
struct Magnitudes {
    uint32_t lo[2], hi[2];
};

// bf16((value(code) * sf) / g) of codes 0..7: the product is exact in binary32, and quotients of magnitudes that are
// powers of two apart are, too (`fast`: nothing leaves the normal range), so two divisions do.
__device__ __forceinline__ Magnitudes magnitudes(float sf, float g, float rcp, bool fast) {
    float v[8];
    if (fast) {
        const float a = div_by_scale(0.5f * sf, g, rcp), b = div_by_scale(1.5f * sf, g, rcp);
        v[0] = 0.0f * a, v[1] = a, v[2] = 2.0f * a, v[3] = b, v[4] = 4.0f * a, v[5] = 2.0f * b, v[6] = 8.0f * a, v[7] = 4.0f * b;
    } else {
        constexpr float kValue[8] = {0.0f, 0.5f, 1.0f, 1.5f, 2.0f, 3.0f, 4.0f, 6.0f};
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = __fdiv_rn(kValue[i] * sf, g);
    }
    Magnitudes m;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const uint32_t p = pack_bf16x2(v[4 * i], v[4 * i + 1]), q = pack_bf16x2(v[4 * i + 2], v[4 * i + 3]);
        m.lo[i] = __byte_perm(p, q, 0x6420);
        m.hi[i] = __byte_perm(p, q, 0x7531);
    }
    return m;
}

// Four codes (the low 16 bits) as two pairs of bf16. The byte permutation picks by a nibble's low three bits; its fourth
// bit, the sign, makes it spread the picked byte's top bit instead, which turns 0x80 into 0xff.
__device__ __forceinline__ uint2 pick4(const Magnitudes& m, uint32_t codes) {
    const uint32_t c = codes & 0x7777u;
    uint32_t sign;
    asm("prmt.b32 %0, %1, %1, %2;" : "=r"(sign) : "r"(0x80808080u), "r"(codes));
    sign = sign << 7 & 0x80808080u;
    const uint32_t lo = __byte_perm(m.lo[0], m.lo[1], c), hi = __byte_perm(m.hi[0], m.hi[1], c) ^ sign;
    return make_uint2(__byte_perm(lo, hi, 0x5140), __byte_perm(lo, hi, 0x7362));
}

template <int CC, bool SWIZZLED>
__global__ void __launch_bounds__(kQuantThreads) dequantize_kernel(QuantArgs a) {
    pdl_wait();
    constexpr int kStep = kQuantThreads / (4 * CC), kTurns = kQuantRows / kStep;
    for (int64_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
        const QuantPlace p = quant_place<CC>(a, tile);
        const int64_t at = (int64_t(p.g) * a.R + p.r) * a.C + p.c;
        uint2 q[kTurns];
        uint32_t sf[kTurns];
#pragma unroll
        for (int i = 0; i < kTurns; i++) {
            q[i] = make_uint2(0, 0);
            sf[i] = 0;
            if (p.r + i * kStep < a.R && p.c < a.C) {
                q[i] = __ldg(reinterpret_cast<const uint2*>(a.codes + (at + int64_t(i) * kStep * a.C) * 8));
                sf[i] = __ldg(a.sf + sf_index<SWIZZLED>(a, p, p.r + i * kStep));
            }
        }
        const float g = __ldg(a.gs + p.g);
        const bool fast = fabsf(g) > 0x1p-60f && fabsf(g) < 0x1p60f;
        const float rcp = fast ? __frcp_rn(g) : 0.0f;
#pragma unroll
        for (int i = 0; i < kTurns; i++) {
            if (p.r + i * kStep >= a.R || p.c >= a.C) continue;
            const Magnitudes m = magnitudes(e4m3_value(sf[i]), g, rcp, fast);
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const uint2 v = pick4(m, (j < 2 ? q[i].x : q[i].y) >> (16 * (j & 1)));
                w[2 * j] = v.x, w[2 * j + 1] = v.y;
            }
            uint16_t* dst = a.out + (at + int64_t(i) * kStep * a.C) * 16;
            if (a.wide) {
                st_v8(dst, w);
            } else {
                st_v4(dst, make_uint4(w[0], w[1], w[2], w[3]));
                st_v4(dst + 8, make_uint4(w[4], w[5], w[6], w[7]));
            }
        }
    }
}

// 64 columns a tile while that keeps the tiles below four for each SM, 256 above: 128 x 7168 then has 112 tiles
// instead of 28, and large matrices read 512 contiguous bytes of a row.
template <typename Kernel>
cudaError_t launch_quant(const LaunchCtx& ctx, QuantArgs a, int64_t G, Kernel narrow, Kernel broad) {
    a.row_tiles = (a.R + 127) / 128 * (128 / kQuantRows);  // the padding rows of the tiles too
    const bool few = G * a.row_tiles * ((a.C + 3) / 4) <= 4 * int64_t(ctx.num_sms);
    a.chunks = few ? (a.C + 3) / 4 : (a.C + 15) / 16;
    a.tiles = G * a.row_tiles * a.chunks;
    return launch_pdl(ctx, few ? narrow : broad, dim3(unsigned(std::min<int64_t>(a.tiles, 1 << 24))),
                      dim3(kQuantThreads), 0, a);
}

}  // namespace

cudaError_t launch_quantize_nvfp4(const LaunchCtx& ctx, const uint16_t* x, int64_t G, int64_t R, int H,
                                  const float* gs, int scale_layout, uint8_t* codes, uint8_t* scales) {
    const QuantArgs a{x, nullptr, codes, scales, gs, 0, int(R), H / 16, 0, 0, reinterpret_cast<uintptr_t>(x) % 32 == 0,
                      H % 64 == 0 && reinterpret_cast<uintptr_t>(scales) % 4 == 0};
    if (scale_layout == MOE_SCALES_SWIZZLED_128X4)
        return launch_quant(ctx, a, G, quantize_kernel<1, true>, quantize_kernel<4, true>);
    return launch_quant(ctx, a, G, quantize_kernel<1, false>, quantize_kernel<4, false>);
}

cudaError_t launch_dequantize_nvfp4(const LaunchCtx& ctx, const uint8_t* codes, const uint8_t* scales, int64_t G,
                                    int64_t R, int H, const float* gs, int scale_layout, uint16_t* out) {
    const QuantArgs a{nullptr, out, const_cast<uint8_t*>(codes), const_cast<uint8_t*>(scales), gs, 0, int(R), H / 16,
                      0, 0, reinterpret_cast<uintptr_t>(out) % 32 == 0, false};
    if (scale_layout == MOE_SCALES_SWIZZLED_128X4)
        return launch_quant(ctx, a, G, dequantize_kernel<1, true>, dequantize_kernel<4, true>);
    return launch_quant(ctx, a, G, dequantize_kernel<1, false>, dequantize_kernel<4, false>);
}

}  // namespace moe
