// Types and arithmetic shared by the kernels over token rows: vectors of a
// row's elements, pairs of fp32 (two lanes of one instruction), softplus and
// the sigmoid.
#pragma once

#include <atomic>

#include "common.cuh"

namespace ofrl {

template <typename T>
__device__ __forceinline__ float to_float(T x) {
    if constexpr (sizeof(T) == 4)
        return x;
    else
        return __bfloat162float(x);
}
template <typename T>
__device__ __forceinline__ T from_float(float x) {
    if constexpr (sizeof(T) == 4)
        return x;
    else
        return __float2bfloat16_rn(x);
}

// V consecutive elements of a row (aligned to their own size), as one load.
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T v[V];
};
template <typename T, int V>
__device__ __forceinline__ void load_vec(float (&out)[V], const T* p) {
    const Vec<T, V> u = *reinterpret_cast<const Vec<T, V>*>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = to_float(u.v[i]);
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&x)[V]) {
    Vec<T, V> u;
#pragma unroll
    for (int i = 0; i < V; ++i) u.v[i] = from_float<T>(x[i]);
    *reinterpret_cast<Vec<T, V>*>(p) = u;
}

// ---- pairs of fp32 -------------------------------------------------------------
using f2 = unsigned long long;
__device__ __forceinline__ f2 f2_of(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f2_split(f2 x, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ float f2_sum(f2 x) {
    float lo, hi;
    f2_split(x, lo, hi);
    return lo + hi;
}
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float exp2_of(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ f2 f2_exp2(f2 x) {
    float lo, hi;
    f2_split(x, lo, hi);
    return f2_of(exp2_of(lo), exp2_of(hi));
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// ---- gates -----------------------------------------------------------------------
// log(1 + e^v) = max(v, 0) + log1p(u), u = e^-|v| in [0, 1]; log1p(u) / u by a
// polynomial fitted here to a relative error of 5e-9 over that range, so small
// steps keep all their bits (log(1 + u) would not).
__device__ __forceinline__ float softplus(float v) {
    const float u = expf(-fabsf(v));
    float p = -0.003244024235755205f;
    p = fmaf(p, u, 0.019851457327604294f);
    p = fmaf(p, u, -0.056959524750709534f);
    p = fmaf(p, u, 0.10603654384613037f);
    p = fmaf(p, u, -0.15305592119693756f);
    p = fmaf(p, u, 0.1967593878507614f);
    p = fmaf(p, u, -0.24954134225845337f);
    p = fmaf(p, u, 0.3332996368408203f);
    p = fmaf(p, u, -0.4999990165233612f);
    p = fmaf(p, u, 1.0f);
    return fmaf(p, u, fmaxf(v, 0.0f));
}
__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.0f, 1.0f + expf(-v)); }

// Opt a kernel into its dynamic shared memory and the largest carveout, once
// per device (the calls cost a few microseconds).
template <typename K>
inline cudaError_t opt_in_once(K kernel, int smem, std::atomic<uint64_t>& done) {
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (device & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    if (smem > 48 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = set_max_shared_carveout(kernel);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

}  // namespace ofrl
