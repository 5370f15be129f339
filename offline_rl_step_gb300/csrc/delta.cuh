// Shared declarations of the sequence-memory kernels (gated delta rule) and
// their context.
#pragma once

#include <atomic>

#include "common.cuh"

struct ofrl_delta {
    int device;
    int num_sms;
    ofrl_delta_shape shape;
    int64_t max_tokens;
    int32_t max_episodes;
    int32_t backward;
    void* base;          // the single cudaMalloc of the context
    int64_t bytes;
    int32_t* status;     // [OFRL_STAT_WORDS]
    unsigned* counter;   // work counter of the gradient kernel
    uint8_t* scratch;    // what lies between the launches of one call
    uint8_t* parts;      // of a forward pass over parts of episodes
};

namespace ofrl {
namespace delta {

constexpr int kChunk = 64;          // tokens per chunk
constexpr int kMaxDim = 128;

// Chunk c of episode e has slot start(e) / 64 + e + c: distinct for distinct
// chunks, and computable from the ends alone (ceil(len / 64) is at most
// end / 64 - start / 64 + 1).
__host__ __device__ inline int64_t slots_of(int64_t tokens, int64_t episodes) { return tokens / kChunk + episodes; }

struct Span {
    int32_t start, len;
};

// Token range of episode e.  Whatever the ends hold, the range lies in
// [0, tokens) and its chunks' slots below slots_of(); ranges of ends that
// ascend do not overlap.
__device__ __forceinline__ Span span_of(const int32_t* ends, int32_t e, int32_t tokens) {
    const int32_t lo = e > 0 ? min(max(ends[e - 1], 0), tokens) : 0;
    const int32_t hi = min(max(ends[e], lo), tokens);
    return {lo, hi - lo};
}
__device__ __forceinline__ bool span_bad(const int32_t* ends, int32_t e, int32_t tokens) {
    const int32_t lo = e > 0 ? ends[e - 1] : 0;
    return ends[e] < lo || ends[e] > tokens;
}

struct SeqLaunch {
    ofrl_delta_shape shape;
    ofrl_delta_tokens in;
    const int32_t* ends;
    int32_t episodes;
    const float* init;
    void* out;
    float* final_state;
    uint8_t* saved;
    const void* dout;
    const float* d_final;
    ofrl_delta_grads grads;
    float* d_init;
    uint8_t* scratch;
    uint8_t* parts;
    unsigned* counter;
    int32_t* status;
    int num_sms;
};

// Threads of a CTA that goes token by token, and the state rows it has there
// with `lanes` lanes to a row, two rows to a lane group.
constexpr int kStepThreads = 128, kRecurRows = 2;
constexpr int recur_rows(int lanes) { return kStepThreads / lanes * kRecurRows; }

struct StepLaunch {
    ofrl_delta_shape shape;
    ofrl_delta_tokens in;
    const int32_t* slot_idx;
    int32_t slots;
    const float* state_in;
    float* state_out;
    void* out;
    int32_t* status;
    int num_sms;
};

// Opt a kernel into its dynamic shared memory and the largest carveout, once
// per device (the calls cost a few microseconds).
template <typename K>
inline cudaError_t opt_in(K kernel, int smem, std::atomic<uint64_t>& done) {
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (device & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = set_max_shared_carveout(kernel);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

cudaError_t launch_forward(const SeqLaunch& a, cudaStream_t st);
cudaError_t launch_backward(const SeqLaunch& a, cudaStream_t st);
cudaError_t launch_recur(const SeqLaunch& a, cudaStream_t st);      // forward, token by token
cudaError_t launch_step(const StepLaunch& a, cudaStream_t st);
int64_t saved_bytes(const ofrl_delta_shape& s, int64_t tokens, int64_t episodes);
int64_t parts_bytes(const ofrl_delta_shape& s, int64_t tokens, int num_sms);
int64_t scratch_bytes(const ofrl_delta_shape& s, int64_t tokens, int64_t episodes, bool backward);

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// exp(g) is exactly zero below this, so clamping changes no decay and keeps
// sums of log decays finite.
constexpr float kMinLogDecay = -110.0f;

}  // namespace delta
}  // namespace ofrl
