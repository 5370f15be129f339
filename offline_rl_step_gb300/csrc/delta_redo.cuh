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

// x[cols][rows] floats as an image of `planes` planes, its columns in slices of SG groups.
__device__ __forceinline__ void put_image(const Redo& a, uint8_t* img, const float* x, int cols, int SG, float up) {
    const int rows = a.rows, RG = rows / 8;
#pragma unroll 1
    for (int i = a.tid; i < rows * cols; i += a.threads) {
        const int r = i % rows, c = i / rows, cg = c / 8;
        float y = nan_if_not_finite(x[i]) * up;
        uint8_t* to = img + ((cg / SG * RG + r / 8) * SG + cg % SG) * kTile + (r & 7) * 16 + (c & 7) * 2;
#pragma unroll 1
        for (int n = 0; n < a.planes; ++n) {
            const __half h = __float2half_rn(y);
            *reinterpret_cast<__half*>(to + (int64_t)n * rows * cols * 2) = h;
            y -= __half2float(h);
        }
    }
}

// By the whole CTA, in shared memory: the state [DK][rows], U [64][rows] and a
// few tokens.  A thread has a row, which goes through shared memory twice a token:
// 3 us of latency with 128 key channels, 1.5 with 64 (a warp to 16 rows, with the
// sums over lanes, took 10).
constexpr int kRedoTokens = 8;
template <int DK>
constexpr int redo_bytes(int rows) {
    return (rows * (DK + kChunk) + kRedoTokens * (2 * DK + rows + 4)) * 4;
}
template <typename T, int DK>
__device__ __forceinline__ void redo_rows(const Redo& a, float* state) {
    __shared__ float red;
    const int rows = a.rows;
    float *u = state + rows * DK, *kq = u + rows * kChunk, *vs = kq + kRedoTokens * 2 * DK, *gb = vs + kRedoTokens * rows;
#pragma unroll 1
    for (int i = a.tid; i < rows * DK; i += a.threads) {
        const int r = a.row0 + i % rows, c = i / rows;
        state[i] = a.first != nullptr && r < a.dv && c < a.dk ? a.first[(int64_t)r * a.dk + c] : 0.0f;
    }
    __syncthreads();
#pragma unroll 1
    for (int t0 = 0; t0 < a.sp.len; t0 += kChunk) {
        const int64_t at = (int64_t)(t0 / kChunk) * a.v_heads;      // images of the chunk, in heads
        const int len = min(kChunk, a.sp.len - t0);
        if (a.state_img != nullptr) {
            const float up = scale_up(cta_most(a, state, rows * DK, &red));
            put_image(a, a.state_img + at * a.planes * rows * DK * 2, state, DK, a.planes == 2 ? kSliceCols / 8 : 1, up);
            if (a.tid == 0) a.state_unit[at] = pow2_inv(up);
#pragma unroll 1
            for (int i = a.tid; i < rows * kChunk; i += a.threads) u[i] = 0.0f;
        }
#pragma unroll 1
        for (int b0 = t0; b0 < t0 + len; b0 += kRedoTokens) {
            __syncthreads();      // the tokens before are done with
            const int n = min(kRedoTokens, t0 + len - b0);
            const int64_t tok = (int64_t)a.sp.start + b0;
#pragma unroll 1
            for (int i = a.tid; i < n * 2 * DK; i += a.threads) {      // keys and queries
                const int j = i / (2 * DK), c = i % DK;
                const bool isq = i / DK % 2 != 0;
                const T* p = isq ? static_cast<const T*>(a.in->q) + (tok + j) * a.in->q_stride
                                 : static_cast<const T*>(a.in->k) + (tok + j) * a.in->k_stride;
                kq[i] = c < a.dk ? to_f(p[(int64_t)a.khead * a.dk + c]) : 0.0f;
            }
#pragma unroll 1
            for (int i = a.tid; i < n * rows; i += a.threads) {
                const int j = i / rows, r = a.row0 + i % rows;
                vs[i] = r < a.dv ? to_f(static_cast<const T*>(a.v)[(tok + j) * a.v_stride + (int64_t)a.head * a.dv + r]) : 0.0f;
            }
            if (a.tid < n) {
                const int64_t t = tok + a.tid;
                float* x = gb + 4 * a.tid;
                x[0] = expf(to_f(static_cast<const T*>(a.in->g)[t * a.in->g_stride + a.head]));
                x[1] = to_f(static_cast<const T*>(a.in->beta)[t * a.in->beta_stride + a.head]);
                if (a.state_img != nullptr)
                    x[2] = pow2_inv(reinterpret_cast<const float*>(a.pairs + at * kPairBytes + 2 * kSquare)[V_KINV * kChunk + b0 - t0 +
                                                                                                         a.tid]);
            }
            __syncthreads();
            if (a.tid >= rows || a.row0 + a.tid >= a.dv) continue;
            float* s = state + a.tid;
#pragma unroll 1
            for (int j = 0; j < n; ++j) {
                const float *k = kq + j * 2 * DK, *q = k + DK;
                const float decay = gb[4 * j], beta = gb[4 * j + 1];
                float sk[4] = {}, sq[4] = {}, kk[4] = {};
#pragma unroll 2
                for (int c = 0; c < a.dk; c += 4) {      // what lies beyond is zero, also beside infinities
                    const float4 k4 = *reinterpret_cast<const float4*>(k + c), q4 = *reinterpret_cast<const float4*>(q + c);
                    const float kz[4] = {k4.x, k4.y, k4.z, k4.w}, qz[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const float x = s[(c + z) * rows];
                        sk[z] += x * kz[z];
                        sq[z] += x * qz[z];
                        kk[z] += kz[z] * qz[z];
                    }
                }
                const float x = beta * (vs[j * rows + a.tid] - decay * ((sk[0] + sk[1]) + (sk[2] + sk[3])));
#pragma unroll 2
                for (int c = 0; c < a.dk; c += 4) {
                    const float4 k4 = *reinterpret_cast<const float4*>(k + c);
                    const float kz[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                    for (int z = 0; z < 4; ++z) s[(c + z) * rows] = decay * s[(c + z) * rows] + x * kz[z];
                }
                if (b0 + j >= a.skip)
                    static_cast<T*>(a.out)[(tok + j) * a.out_stride + (int64_t)a.head * a.dv + a.row0 + a.tid] = from_f<T>(
                        a.in->scale * (decay * ((sq[0] + sq[1]) + (sq[2] + sq[3])) + x * ((kk[0] + kk[1]) + (kk[2] + kk[3]))));
                if (a.state_img != nullptr) u[(b0 + j - t0) * rows + a.tid] = gb[4 * j + 2] * x;
            }
        }
        __syncthreads();
        if (a.state_img != nullptr) {
            const float up = scale_up(cta_most(a, u, rows * kChunk, &red));
            put_image(a, a.vec_img + at * a.planes * rows * kChunk * 2, u, kChunk, a.planes == 2 ? 8 : 1, up);
            if (a.tid == 0) a.vec_unit[at] = pow2_inv(up);
            __syncthreads();
        }
    }
    if (a.last != nullptr)
#pragma unroll 1
        for (int i = a.tid; i < rows * DK; i += a.threads) {
            const int r = a.row0 + i % rows, c = i / rows;
            if (r < a.dv && c < a.dk) a.last[(int64_t)r * a.dk + c] = state[i];
        }
}

}  // namespace delta
}  // namespace ofrl
