// moe_host.h -- host-side helpers of the extern "C" entry points (moe_abi.cu, experts_abi.cu).
#pragma once

#include <climits>
#include <cstdint>
#include <cuda_runtime.h>

#include "moe_dispatch.h"
#include "moe_launch.h"

namespace moe {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline moe_status_t make_ctx(moe_stream_t stream, LaunchCtx* ctx) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return MOE_ERR_CUDA;
    ctx->stream = reinterpret_cast<cudaStream_t>(stream);
    ctx->num_sms = sms > 0 ? sms : 1;
    ctx->device = dev;
    return MOE_OK;
}

inline moe_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// shared checks of (T, K, E)
inline moe_status_t check_shape(int64_t T, int K, int E) {
    if (T < 0) return MOE_ERR_INVALID_ARG;
    if (K < 1 || E < 1) return MOE_ERR_INVALID_ARG;
    if (K > MOE_MAX_TOPK || E > MOE_MAX_EXPERTS) return MOE_ERR_UNSUPPORTED;
    if (T > 0 && T > int64_t(INT32_MAX) / K) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

}  // namespace moe
