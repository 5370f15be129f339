// Argument checks shared by the operators over token rows.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace ofrl {

inline bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline int64_t dtype_size(int32_t dtype) { return dtype == OFRL_DTYPE_F32 ? 4 : 2; }
inline bool dtype_ok(int32_t dtype) { return dtype == OFRL_DTYPE_F32 || dtype == OFRL_DTYPE_BF16; }
// Tokens of a call, at most: an index may run a CTA's tokens past them.
constexpr int64_t kMaxTokens = ((int64_t)1 << 31) - ((int64_t)1 << 17);
inline bool counts_ok(int64_t tokens, int64_t episodes) {
    return tokens >= 0 && tokens <= kMaxTokens && episodes >= 0 && episodes <= INT32_MAX;
}
// Rows of `width` elements: at least that far apart, addressable.
inline bool stride_ok(int64_t stride, int64_t width) { return stride >= width && stride <= (int64_t)1 << 40; }
// A buffer of 16-byte rows.
inline bool rows_ok(const void* p, int64_t stride, int64_t width, int64_t elem) {
    return p != nullptr && aligned_to(p, 16) && stride_ok(stride, width) && stride * elem % 16 == 0;
}
inline ofrl_status cuda_status(cudaError_t e) { return e == cudaSuccess ? OFRL_OK : OFRL_ECUDA; }
// The context's device must be the current one.
template <typename Ctx>
inline ofrl_status check_device(const Ctx* ctx) {
    if (ctx == nullptr) return OFRL_EINVAL;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return OFRL_ECUDA;
    return dev == ctx->device ? OFRL_OK : OFRL_EINVAL;
}
// The current device and how many SMs it has (0: none).
inline int current_sms(int* device) {
    int sms = 0;
    if (cudaGetDevice(device) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, *device) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return sms;
}
template <typename Ctx>
inline ofrl_status poll_words(Ctx* ctx, void* stream, int32_t* words_out) {
    const ofrl_status s = check_device(ctx);
    if (s != OFRL_OK) return s;
    if (words_out == nullptr) return OFRL_EINVAL;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemcpyAsync(words_out, ctx->status, OFRL_STAT_WORDS * 4, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaMemsetAsync(ctx->status, 0, OFRL_STAT_WORDS * 4, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    return cuda_status(e);
}
// One allocation of `bytes`, its first OFRL_STAT_WORDS words zero.
inline cudaError_t take_memory(void** base, int64_t bytes) {
    cudaError_t e = cudaMalloc(base, (size_t)bytes);
    if (e == cudaSuccess) {
        e = cudaMemset(*base, 0, OFRL_STAT_WORDS * 4);
        if (e == cudaSuccess) e = cudaDeviceSynchronize();
        if (e != cudaSuccess) cudaFree(*base);
    }
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}
template <typename Ctx>
inline ofrl_status release_memory(Ctx* ctx) {
    if (ctx == nullptr) return OFRL_OK;
    const cudaError_t e1 = cudaDeviceSynchronize(), e2 = cudaFree(ctx->base);
    delete ctx;
    return e1 == cudaSuccess && e2 == cudaSuccess ? OFRL_OK : OFRL_ECUDA;
}

}  // namespace ofrl
