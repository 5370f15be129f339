// Types and arithmetic shared by the kernels over token rows: vectors of a
// row's elements, pairs of fp32 (two lanes of one instruction), softplus and
// the sigmoid.
#pragma once

#include <atomic>
#include <cmath>

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

// Asynchronous copies of BYTES (4, 8 or 16) to shared memory, in groups.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
    const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// Asks for `bytes` (a multiple of 16, 16-byte aligned) to be brought into L2.
__device__ __forceinline__ void prefetch_l2(const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
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
__device__ __forceinline__ float f2_lo(f2 x) {
    float lo, hi;
    f2_split(x, lo, hi);
    return lo;
}
__device__ __forceinline__ float f2_hi(f2 x) {
    float lo, hi;
    f2_split(x, lo, hi);
    return hi;
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

// Elements 2 i and 2 i + 1 of a raw vector, and a vector from pairs.
template <typename T, int V>
__device__ __forceinline__ f2 vec_pair(const Vec<T, V>& u, int i) {
    if constexpr (sizeof(T) == 2) {
        const uint32_t w = reinterpret_cast<const uint32_t*>(u.v)[i];
        return f2_of(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    } else {
        return f2_of(u.v[2 * i], u.v[2 * i + 1]);
    }
}
template <typename T, int V>
__device__ __forceinline__ void set_vec_pair(Vec<T, V>& u, int i, f2 x) {
    if constexpr (sizeof(T) == 2) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f2_lo(x), f2_hi(x));
        reinterpret_cast<uint32_t*>(u.v)[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
        u.v[2 * i] = f2_lo(x);
        u.v[2 * i + 1] = f2_hi(x);
    }
}

// ---- gates -----------------------------------------------------------------------
__device__ __forceinline__ f2 f2_add(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 f2_both(float x) { return f2_of(x, x); }
// What a state is multiplied by, exp2(delta A2).  A slow state is multiplied by
// thousands of these, so their mean error counts and not each one's rounding: that
// of ex2.approx, measured over exponents of -2^-16 .. -1, is -5e-9 .. -2.7e-8 of the
// value, and its rounding 3e-8.  With this added to the exponent, which the product
// takes along for nothing, it is within 1.3e-8 of zero (dA of 65 thousand tokens:
// 1.2e-6 off, then 7.8e-7).  Steps of zero still give exactly 1.
constexpr float kDecayBias = 2e-8f;
__device__ __forceinline__ float decay_of(float delta, float a2) { return exp2_of(fmaf(delta, a2, kDecayBias)); }
__device__ __forceinline__ f2 f2_decay(f2 delta, f2 a2) { return f2_exp2(f2_fma(delta, a2, f2_both(kDecayBias))); }
__device__ __forceinline__ float rcp_of(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float max_or_nan(float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}

// log(1 + e^v) = max(v, 0) + log1p(u), u = e^-|v| in [0, 1]; log1p(u) / u by a
// polynomial fitted here, one coefficient after the other rounded to fp32 and held
// while the rest were fitted again: 5.4e-9 of the value off over that range, so small
// steps keep all their bits (log(1 + u) would not).  u is 2^x with what rounding
// x = -|v| log2 e leaves put back, or far steps would lose bits; with it goes part of
// ex2.approx's mean error, -5e-8 of the value below 2^-1, -2e-8 above (measured).  More
// than 2.9e-8 would round values above 2^-1 up.  What is left in a step's mean error is
// at most 2.6e-8 (without: 5.4e-8).
constexpr float kExp2Mean = 2.8e-8f;
__device__ __forceinline__ f2 softplus(f2 v, f2& u) {
    float a, b, lo, hi;
    f2_split(v, a, b);
    // below -200, u is zero anyway and infinities would leave a rest that is no number
    const f2 n = f2_of(fmaxf(-fabsf(a), -200.0f), fmaxf(-fabsf(b), -200.0f));
    const f2 x = f2_mul(n, f2_both(kLog2e));
    f2_split(x, lo, hi);
    f2 rest = f2_fma(n, f2_both(kLog2e), f2_of(-lo, -hi));
    rest = f2_fma(n, f2_both(1.92596299e-8f), rest);      // log2 e less its fp32 value
    u = f2_of(exp2_of(lo), exp2_of(hi));
    u = f2_fma(u, f2_fma(rest, f2_both(kLn2), f2_both(kExp2Mean)), u);
    f2 p = f2_both(-0.0033244711812585592f);
    p = f2_fma(p, u, f2_both(0.02023317851126194f));
    p = f2_fma(p, u, f2_both(-0.05772183835506439f));
    p = f2_fma(p, u, f2_both(0.1068684533238411f));
    p = f2_fma(p, u, f2_both(-0.1535947173833847f));
    p = f2_fma(p, u, f2_both(0.19696977734565735f));
    p = f2_fma(p, u, f2_both(-0.24958936870098114f));
    p = f2_fma(p, u, f2_both(0.3333055078983307f));
    p = f2_fma(p, u, f2_both(-0.49999934434890747f));
    p = f2_fma(p, u, f2_both(1.0f));
    return f2_fma(p, u, f2_of(max_or_nan(a, 0.0f), max_or_nan(b, 0.0f)));
}
__device__ __forceinline__ f2 softplus(f2 v) {
    f2 u;
    return softplus(v, u);
}
// softplus and its slope, the sigmoid: 1 / (1 + u) or u / (1 + u).
__device__ __forceinline__ f2 softplus_slope(f2 v, f2& slope) {
    f2 u;
    const f2 y = softplus(v, u), e = f2_add(u, f2_both(1.0f));
    const float r0 = rcp_of(f2_lo(e)), r1 = rcp_of(f2_hi(e));
    slope = f2_of(f2_lo(v) < 0.0f ? f2_lo(u) * r0 : r0, f2_hi(v) < 0.0f ? f2_hi(u) * r1 : r1);
    return y;
}
// 1 / (1 + e^-v): a few 2^-22 off up to |v| of 8 or so, where it matters.
__device__ __forceinline__ f2 sigmoid(f2 v) {
    const f2 e = f2_add(f2_exp2(f2_mul(v, f2_both(-kLog2e))), f2_both(1.0f));
    return f2_of(rcp_of(f2_lo(e)), rcp_of(f2_hi(e)));
}
__device__ __forceinline__ float sigmoid(float v) { return rcp_of(1.0f + exp2_of(-kLog2e * v)); }
__device__ __forceinline__ float softplus(float v) { return f2_lo(softplus(f2_of(v, v))); }
// v sigmoid(v), and its slope s (1 + v (1 - s)) given s = sigmoid(v).
__device__ __forceinline__ f2 silu(f2 v) { return f2_mul(v, sigmoid(v)); }
__device__ __forceinline__ f2 silu_slope(f2 v, f2 s) {
    return f2_fma(f2_mul(v, s), f2_fma(s, f2_both(-1.0f), f2_both(1.0f)), s);
}

// Opt a kernel into its dynamic shared memory and the largest carveout, once
// per device (the calls cost a few microseconds).
template <typename K>
inline cudaError_t opt_in_once(K kernel, int smem, std::atomic<uint64_t>& done) {
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (device & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    if (smem > 40 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = set_max_shared_carveout(kernel);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

}  // namespace ofrl
