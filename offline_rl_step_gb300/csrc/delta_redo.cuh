// What a chain does for an episode with tokens or states that are not finite,
// or with a chunk within which states grow beyond its operands' range (the
// preparing kernel makes such a chunk's x NaN).
//
// The zeros of T and P are multiplied like everything else, so within a chunk a
// NaN or an infinity reaches the tokens before it.  Where v, k, g or beta of a
// token, or the state before it, is not finite, u is not either, and u k^T then
// leaves no element of the state's row finite, for good (a decay of zero does not
// clear a NaN).  So a chain looks at an element of each row once, at its end (on
// tcgen05, where the last state is not made, at every chunk's largest u), and a
// CTA that finds one not finite goes over its rows of the episode again, token by
// token as the recurrence is written, and replaces what it left.  A q that is not
// finite stays with its token.
//
// What this costs calls that have nothing of the kind: 64 episodes of 256 tokens
// 26.3 us with and without, about 65k ragged transitions learn 589 us against 583,
// 32768 tokens in parts 350 against 347.  Sealing such channels within the pass
// cost 7 to 13% of it.
#pragma once

#include "delta_mma.cuh"

namespace ofrl {
namespace delta {

struct Redo {
    int tid, threads;
    const ofrl_delta_tokens* in;
    const void* v;                  // of token 0
    void* out;
    int64_t v_stride, out_stride;
    Span sp;
    int skip;                       // tokens whose outputs are there already
    int head, khead, v_heads, dk, dv;
    int row0, rows;                 // the CTA's first row, and how many it has
    const float* first;             // the episode's and head's state, or null
    float* last;                    // where its state goes afterwards, or null
    // images for the gradients, or null
    uint8_t *state_img, *vec_img;   // of the first chunk and this head
    float *state_unit, *vec_unit;
    const uint8_t* pairs;
    int planes;
};

// Registers of the block and the thread read anew: what a pass worked out of
// them is not to be kept for what comes after it.
__device__ __forceinline__ unsigned fresh_block() {
    unsigned x;
    asm volatile("mov.u32 %0, %%ctaid.x;" : "=r"(x));
    return x;
}
__device__ __forceinline__ unsigned fresh_thread() {
    unsigned x;
    asm volatile("mov.u32 %0, %%tid.x;" : "=r"(x));
    return x;
}

// NaN for what is not finite: it is left out of largest magnitudes.
__device__ __forceinline__ float nan_if_not_finite(float x) { return isfinite(x) ? x : NAN; }

// Largest finite magnitude of n floats in shared memory, by the whole CTA;
// red: a float in shared memory.
__device__ __forceinline__ float cta_most(const Redo& a, const float* x, int n, float* red) {
    float m = 0.0f;
#pragma unroll 1
    for (int i = a.tid; i < n; i += a.threads)
        if (isfinite(x[i])) m = fmaxf(m, fabsf(x[i]));
    if (a.tid == 0) *red = 0.0f;
    __syncthreads();
    atomicMax(reinterpret_cast<int*>(red), __float_as_int(m));      // magnitudes are ordered as integers
    __syncthreads();
    m = *red;
    __syncthreads();
    return m;
}

// [rows][cols] floats as an image of `planes` planes, its columns in slices of SG groups.
__device__ __forceinline__ void put_image(const Redo& a, uint8_t* img, const float* x, int rows, int cols, int SG, int planes, float up) {
    const int RG = rows / 8;
#pragma unroll 1
    for (int i = a.tid; i < rows * cols; i += a.threads) {
        const int r = i / cols, c = i % cols, cg = c / 8;
        float y = nan_if_not_finite(x[i]) * up;
        uint8_t* to = img + ((cg / SG * RG + r / 8) * SG + cg % SG) * kTile + (r & 7) * 16 + (c & 7) * 2;
#pragma unroll 1
        for (int n = 0; n < planes; ++n) {
            const __half h = __float2half_rn(y);
            *reinterpret_cast<__half*>(to + (int64_t)n * rows * cols * 2) = h;
            y -= __half2float(h);
        }
    }
}

// By the whole CTA, over state[rows][DK] and, for images, u[rows][64] in shared
// memory.  Nothing here is fast.
template <typename T, int DK>
__device__ __forceinline__ void redo_rows(const Redo& a, float* state, float* u) {
    __shared__ float red;
    const int warp = a.tid >> 5, lane = a.tid & 31, warps = a.threads >> 5;
#pragma unroll 1
    for (int i = a.tid; i < a.rows * DK; i += a.threads) {
        const int r = a.row0 + i / DK, c = i % DK;
        float x = 0.0f;
        if (a.first != nullptr && r < a.dv && c < a.dk)
            x = a.first[(int64_t)r * a.dk + c];
        state[i] = x;
    }
    __syncthreads();
    for (int t0 = 0; t0 < a.sp.len; t0 += kChunk) {
        const int64_t at = (int64_t)(t0 / kChunk) * a.v_heads;      // images of the chunk, in heads
        const int len = min(kChunk, a.sp.len - t0);
        if (a.state_img != nullptr) {
            const float up = scale_up(cta_most(a, state, a.rows * DK, &red));
            put_image(a, a.state_img + at * a.planes * a.rows * DK * 2, state, a.rows, DK, a.planes == 2 ? kSliceCols / 8 : 1,
                      a.planes, up);
            if (a.tid == 0) a.state_unit[at] = pow2_inv(up);
#pragma unroll 1
            for (int i = a.tid; i < a.rows * kChunk; i += a.threads) u[i] = 0.0f;
            __syncthreads();
        }
        for (int t = t0; t < t0 + len; ++t) {
            const int64_t tok = (int64_t)a.sp.start + t;
            const T* k = static_cast<const T*>(a.in->k) + tok * a.in->k_stride + (int64_t)a.khead * a.dk;
            const T* q = static_cast<const T*>(a.in->q) + tok * a.in->q_stride + (int64_t)a.khead * a.dk;
            const float decay = expf(to_f(static_cast<const T*>(a.in->g)[tok * a.in->g_stride + a.head]));
            const float beta = to_f(static_cast<const T*>(a.in->beta)[tok * a.in->beta_stride + a.head]);
            const float kappa =
                a.state_img == nullptr
                    ? 0.0f
                    : pow2_inv(reinterpret_cast<const float*>(a.pairs + at * kPairBytes + 2 * kSquare)[V_KINV * kChunk + t - t0]);
#pragma unroll 1
            for (int r = warp; r < a.rows; r += warps) {
                const int row = a.row0 + r;
                if (row >= a.dv) break;      // no row: zero, and stays so
                float* s = state + r * DK;
                float sk = 0.0f, sq = 0.0f, kq = 0.0f;
#pragma unroll 1
                for (int c = lane; c < a.dk; c += 32) {      // what lies beyond is zero, also beside infinities
                    const float kc = to_f(k[c]), qc = to_f(q[c]);
                    sk += s[c] * kc;
                    sq += s[c] * qc;
                    kq += kc * qc;
                }
                sk = warp_sum(sk);
                sq = warp_sum(sq);
                kq = warp_sum(kq);
                const float v = to_f(static_cast<const T*>(a.v)[tok * a.v_stride + (int64_t)a.head * a.dv + row]);
                const float x = beta * (v - decay * sk);
#pragma unroll 1
                for (int c = lane; c < a.dk; c += 32) s[c] = decay * s[c] + x * to_f(k[c]);
                if (lane == 0) {
                    if (t >= a.skip)
                        static_cast<T*>(a.out)[tok * a.out_stride + (int64_t)a.head * a.dv + row] =
                            from_f<T>(a.in->scale * (decay * sq + x * kq));
                    if (a.state_img != nullptr) u[r * kChunk + t - t0] = kappa * x;
                }
            }
        }
        __syncthreads();
        if (a.state_img != nullptr) {
            const float up = scale_up(cta_most(a, u, a.rows * kChunk, &red));
            put_image(a, a.vec_img + at * a.planes * a.rows * kChunk * 2, u, a.rows, kChunk, a.planes == 2 ? 8 : 1, a.planes,
                      up);
            if (a.tid == 0) a.vec_unit[at] = pow2_inv(up);
            __syncthreads();
        }
    }
    if (a.last != nullptr)
        for (int i = a.tid; i < a.rows * DK; i += a.threads) {
            const int r = a.row0 + i / DK, c = i % DK;
            if (r < a.dv && c < a.dk) a.last[(int64_t)r * a.dk + c] = state[i];
        }
}

}  // namespace delta
}  // namespace ofrl
