// Two host threads in one C entry point, one with calls that need little shared memory and one with calls that need much.
// Prints how many calls did not return MOE_OK, of each entry point.
#include <atomic>
#include <cstdio>
#include <functional>
#include <thread>

#include <cuda_runtime.h>

#include "moe_dispatch.h"
#include "moe_experts.h"

namespace {

// Zeroed device memory, never freed: the process ends with the test.
template <typename T>
T* zeros(size_t n) {
    void* p = nullptr;
    if (cudaMalloc(&p, n * sizeof(T)) != cudaSuccess || cudaMemset(p, 0, n * sizeof(T)) != cudaSuccess) std::abort();
    return static_cast<T*>(p);
}

using Call = std::function<moe_status_t(moe_stream_t)>;

Call product(int E) {
    const int M = 2, n = 64, k = 64;
    auto* a = zeros<uint8_t>(size_t(E) * M * k / 2);
    auto* sf = zeros<uint8_t>(size_t(E) * M * k / 16);
    auto* w = zeros<uint8_t>(size_t(E) * n * k / 2);
    auto* wsf = zeros<uint8_t>(size_t(E) * 128 * k / 16);
    auto* count = zeros<int32_t>(E);
    auto* out = zeros<uint16_t>(size_t(E) * M * n);
    auto* status = zeros<int32_t>(1);
    return [=](moe_stream_t s) {
        return moe_expert_gemm(MOE_MODE_MASKED, a, sf, MOE_SCALES_ROW_MAJOR, E, M, 0, n, k, nullptr, count, w, wsf, nullptr, out,
                               status, s);
    };
}

Call layer(int T, int K) {
    const int E = 2, H = 64, I = 64;
    auto* x = zeros<uint16_t>(size_t(T) * H);
    auto* ids = zeros<int32_t>(size_t(T) * K);
    auto* g = zeros<float>(size_t(T) * K);
    auto* w13 = zeros<uint8_t>(size_t(E) * 2 * I * H / 2);
    auto* s13 = zeros<uint8_t>(size_t(E) * 2 * 128 * H / 16);
    auto* w2 = zeros<uint8_t>(size_t(E) * H * I / 2);
    auto* s2 = zeros<uint8_t>(size_t(E) * 128 * I / 16);
    auto* out = zeros<uint16_t>(size_t(T) * H);
    const size_t bytes = moe_layer_workspace_size(T, K, H, I, E);
    auto* ws = zeros<uint8_t>(bytes);
    auto* status = zeros<int32_t>(1);
    return [=](moe_stream_t s) {
        return moe_layer_few_tokens(x, T, H, I, ids, g, K, E, MOE_QUANT_NVFP4_B16, w13, s13, nullptr, w2, s2, nullptr, out, ws,
                                    bytes, status, s);
    };
}

Call route(int E) {
    const int T = 700, K = 4;
    auto* ids = zeros<int32_t>(T * K);
    auto* seg = zeros<int64_t>(E + 1);
    auto* dst = zeros<int32_t>(T * K);
    auto* order = zeros<int32_t>(T * K);
    auto* count = zeros<int32_t>(E);
    auto* parts = zeros<int32_t>(1);
    const size_t bytes = moe_route_meta_workspace_size(T, K, E);
    void* ws = zeros<uint8_t>(bytes + 1);
    auto* status = zeros<int32_t>(1);
    return [=](moe_stream_t s) {
        return moe_route_meta(ids, T, K, E, 1, 0, seg, dst, order, count, parts, nullptr, ws, bytes, status, s);
    };
}

int refused(const Call& little, const Call& much) {
    std::atomic<int> wrong{0}, ready{0};
    auto work = [&](const Call& call) {
        cudaStream_t s;
        if (cudaStreamCreateWithFlags(&s, cudaStreamNonBlocking) != cudaSuccess) std::abort();
        ready++;
        while (ready < 2) {}
        for (int i = 0; i < 10000; i++) {
            if (call(reinterpret_cast<moe_stream_t>(s)) != MOE_OK) wrong++;
            if (i % 100 == 99) cudaStreamSynchronize(s);
        }
        cudaStreamSynchronize(s);
    };
    cudaDeviceSynchronize();
    std::thread a([&] { work(little); }), b([&] { work(much); });
    a.join();
    b.join();
    return wrong;
}

}  // namespace

int main() {
    std::printf("product %d\n", refused(product(4), product(MOE_MAX_EXPERTS)));
    std::printf("layer %d\n", refused(layer(1, 1), layer(64, 16)));
    std::printf("route %d\n", refused(route(500), route(MOE_MAX_EXPERTS)));
    return cudaDeviceSynchronize() == cudaSuccess ? 0 : 1;
}
