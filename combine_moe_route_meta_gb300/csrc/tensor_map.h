// tensor_map.h -- host side of the tensor-map loads.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace moe {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

// A map of bytes [.., d1, d0] (densely packed, d0 a multiple of 16) read in boxes of b1 (x b2 ..) rows of 128
// bytes, which land in the 128-byte swizzle; what is out of range reads as zero.
inline bool make_map(CUtensorMap* map, const void* p, int rank, const uint64_t* dims, const uint32_t* box) {
    if (!encode_tiled()) return false;
    cuuint64_t size[4], stride[3];
    cuuint32_t b[4], one[4] = {1, 1, 1, 1};
    uint64_t bytes = 1;
    for (int i = 0; i < rank; i++) {
        size[i] = dims[i];
        b[i] = box[i];
        bytes *= dims[i];
        if (i + 1 < rank) stride[i] = bytes;
    }
    return encode_tiled()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, cuuint32_t(rank), const_cast<void*>(p), size, stride, b,
                          one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace moe
