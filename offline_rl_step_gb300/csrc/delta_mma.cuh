// Warp-level building blocks of the sequence-memory kernels: mma.sync
// fragments, shared-memory matrix images, and fp16 operands with powers of
// two taken out.
//
// Matrix image: 8x8 blocks of 16-bit elements, each 128 contiguous bytes
// (eight 16-byte rows), block (row group, column group) at
// (row_group * column_groups + column_group) * 128.  ldmatrix reads a block
// without bank conflicts, plain or transposed, and one register of an mma
// accumulator's layout over 32 lanes is exactly one block.
//
// Operands.  A value x becomes fp16 after division by a power of two that
// brings its tile's largest magnitude into [2^13, 2^14): 11 significand bits
// over 27 binades below the largest.  Two planes (x = hi + lo) carry 22 bits.
// Products accumulate in fp32 and the powers of two are multiplied back in
// fp32, so the only roundings are those of the planes.
#pragma once

#include <cuda_fp16.h>

#include "delta.cuh"
#include "umma.cuh"

namespace ofrl {
namespace delta {

constexpr int kTile = 8 * 8 * 2;                 // bytes of an 8x8 block
constexpr int kSquare = kChunk * kChunk * 2;     // bytes of a 64x64 image plane

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void stsm4t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d) : "memory");
}
// d += a b^T: a 16x16 (row), b 16x8 (k x n), fp32 accumulation.
__device__ __forceinline__ void mma_h(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_b(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_h(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_h(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
__device__ __forceinline__ uint32_t pack_b(float x, float y) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_b(uint32_t u) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
}

// N fp16 planes of (x, y): each holds what the ones before left.
template <int N>
__device__ __forceinline__ void planes_h(float x, float y, uint32_t (&p)[N]) {
    p[0] = pack_h(x, y);
    if constexpr (N == 2) {
        const float2 f = unpack_h(p[0]);
        p[1] = pack_h(x - f.x, y - f.y);
    }
}
template <int N>
__device__ __forceinline__ void planes_b(float x, float y, uint32_t (&p)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        p[i] = pack_b(x, y);
        const float2 f = unpack_b(p[i]);
        x -= f.x;
        y -= f.y;
    }
}

// Power of two s with amax * s in [2^13, 2^14) (1 for a non-finite amax, the
// largest for zero: a zero tile then outweighs no other); its inverse is exact.
__device__ __forceinline__ float scale_up(float amax) {
    const int e = (int)((__float_as_uint(amax) >> 23) & 255u);
    return e == 255 ? 1.0f : __uint_as_float((uint32_t)min(267 - e, 252) << 23);
}
// 1 / s of a power of two.
__device__ __forceinline__ float pow2_inv(float s) { return __uint_as_float(0x7F000000u - __float_as_uint(s)); }

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Columns 8 t + 2 (lane & 3), + 1 of vector `which`.
__device__ __forceinline__ float2 vec2(const float* vec, int which, int t) {
    return *reinterpret_cast<const float2*>(vec + which * kChunk + t * 8 + (threadIdx.x & 3) * 2);
}

// Accumulator tiles x[t] (16 rows x 8 columns each, NT of them side by side)
// times s as A operands: N planes of NT/2 fragments.
template <int N, int NT>
__device__ __forceinline__ void to_frags(const float (&x)[NT][4], float s, uint32_t (&a)[N][NT / 2][4]) {
#pragma unroll
    for (int k = 0; k < NT / 2; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float* t = x[2 * k + (i >> 1)] + (i & 1) * 2;
            uint32_t p[N];
            planes_h<N>(t[0] * s, t[1] * s, p);
#pragma unroll
            for (int n = 0; n < N; ++n) a[n][k][i] = p[n];
        }
}

template <int NT>
__device__ __forceinline__ float tile_max(const float (&x)[NT][4]) {
    float m = 0.0f;
#pragma unroll
    for (int t = 0; t < NT; ++t)
        m = fmaxf(m, fmaxf(fmaxf(fabsf(x[t][0]), fabsf(x[t][1])), fmaxf(fabsf(x[t][2]), fabsf(x[t][3]))));
    return warp_max(m);
}

// d[t] += a b for column tiles t0 .. t0 + NT - 1 of the operand B, an image of
// CG column groups in shared memory at `b` (NB planes of `plane` bytes).
// TRANS: the image's rows run along k (else along n).  Planes i of a and j of
// b are multiplied when i + j < max(NA, NB): what is dropped is below 2^-22.
// The tensor cores cut off what a sum cannot hold, so the small products come
// first, for all k, while the sums are small: fp32 gradients of the keys over
// 256 tokens end 4.2e-7 off, 6.0e-7 with all products of a k step together (the
// error lies to one side), for 6% more time from reading plane 0 twice.
// KTO: the k steps of 16 that are taken.  TRI: what B is zero for and need not
// be multiplied, nothing, columns before the row (kUpper) or after it (kLower).
enum Tri { kFull, kUpper, kLower };
template <int KTO, int NT, int NA, int NB, bool TRANS, Tri TRI = kFull, int KA>
__device__ __forceinline__ void gemm(float (&d)[NT][4], const uint32_t (&a)[NA][KA][4], uint32_t b, int plane, int CG,
                                     int t0) {
    const int lane = threadIdx.x & 31;
    const int m = lane >> 3, r = lane & 7;
    constexpr int NP = NA > NB ? NA : NB;
#pragma unroll
    for (int ij = NP - 1; ij >= 0; --ij)
#pragma unroll
        for (int k = 0; k < KTO; ++k)
#pragma unroll
            for (int t = 0; t < NT; t += 2)
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    const int i = ij - j;
                    if (i < 0 || i >= NA || (TRI == kUpper && t < 2 * k) || (TRI == kLower && t > 2 * k + 1)) continue;
                    // matrices 0, 1: k halves of tile t; 2, 3: of tile t + 1
                    const int kg = 2 * k + (m & 1), ng = t0 + t + (m >> 1);
                    const uint32_t at = b + j * plane + (TRANS ? kg * CG + ng : ng * CG + kg) * kTile + r * 16;
                    uint32_t f[4];
                    if (TRANS)
                        ldsm4t(f, at);
                    else
                        ldsm4(f, at);
                    mma_h(d[t], a[i][k], f[0], f[1]);
                    mma_h(d[t + 1], a[i][k], f[2], f[3]);
                }
}

template <int NT>
__device__ __forceinline__ void zero(float (&x)[NT][4]) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[t][i] = 0.0f;
}

// ---- what the preparing kernel leaves per chunk -----------------------------
//
// Keys and queries are divided by powers of two per row, kappa_i and kq_i, so
// that a row's largest magnitude lies in [1, 2).  With k^ = k / kappa, v^ = v /
// kappa, beta^ = beta kappa^2 the recurrence keeps its form and its states, and
// u^ = kappa u; every kernel works on these.
struct KeyImage {      // per (slot, key head): K^ planes, then Q^ planes
    static __host__ __device__ constexpr int64_t bytes(int dk_pad, int planes) {
        return 2LL * planes * kChunk * dk_pad * 2;
    }
};
// Per (slot, value head): (T^T) plane 0, P plane 0, vectors, then planes 1.
// T^T rows j (16 of them share a power of two), columns i, of T = (1 + A)^-1;
// P rows i, columns j, divided by the chunk's unit of P.
constexpr float kPScale = 32.0f;     // |q^ k^| < 4 * 128: P below 2^14 where no decay D_ij is above 1
constexpr int kMost = 0, kPUnit = 1;      // in V_MISC
enum Vec {
    V_GAM,      // gamma
    V_REST,     // exp(G_last - G_j)
    V_BETA,     // beta^
    V_TINV,     // unit of T^T's row
    V_QS,       // scale kq (0 past the chunk's end)
    V_QINV,     // 1 / kq
    V_KINV,     // 1 / kappa
    V_GHI,      // G (log2) as a sum of two floats
    V_GLO,
    V_XV,       // beta^ tinv / kappa: of v in beta x, ready for T^T
    V_XS,       // beta^ tinv gamma: of S k in it
    V_OS,       // scale kq gamma
    V_DV,       // beta^ / kappa
    V_DS,       // beta^ gamma
    V_MISC,     // [0]: the largest of rest and 1; [1]: P's unit
    V_COUNT
};
constexpr int kVecBytes = V_COUNT * kChunk * 4;
constexpr int64_t kPairFirst = 2 * kSquare + kVecBytes;
constexpr int64_t kPairBytes = 4 * kSquare + kVecBytes;

// Padded widths of the instances.
__host__ __device__ inline int pad_dim(int d) { return d <= 64 ? 64 : 128; }
inline int token_planes(int32_t dtype) { return dtype == OFRL_DTYPE_F32 ? 2 : 1; }

struct Prepared {
    uint8_t* keys;
    uint8_t* pairs;
};

// Per (slot, value head): the state before a chunk [v_dim_pad][k_dim_pad] and
// U^T (or R^T) [v_dim_pad][64] as images of token_planes() planes, each with
// one power of two (state_unit, vec_unit).  Images of two planes: the state's
// cut into slices of 32 columns, each contiguous, U^T's with its blocks in row
// order.  Images of one plane: blocks column group by column group.
constexpr int kSliceCols = 32;
struct Images {
    uint8_t* state;
    uint8_t* vec;
    float* state_unit;
    float* vec_unit;
};

// planes: of T and P, and of every intermediate of the forward pass (1 or 2).
cudaError_t launch_prep(const SeqLaunch& a, const Prepared& to, int planes, cudaStream_t st);
cudaError_t launch_chain_forward(const SeqLaunch& a, const Prepared& p, const Images& img, int planes, cudaStream_t st);
cudaError_t launch_chain_forward_tc(const SeqLaunch& a, const Prepared& p, const Images& img, cudaStream_t st);
cudaError_t launch_chain_reverse_tc(const SeqLaunch& a, const Prepared& p, const Images& img, cudaStream_t st);
cudaError_t launch_chain_reverse(const SeqLaunch& a, const Prepared& p, const Images& img, cudaStream_t st);
cudaError_t launch_grad_tc(const SeqLaunch& a, const Prepared& p, const Images& fwd, const Images& rev, cudaStream_t st);
cudaError_t launch_grad(const SeqLaunch& a, const Prepared& p, const Images& fwd, const Images& rev, cudaStream_t st);

// The chunk of a slot.
struct Chunk {
    int64_t tok;      // its first token
    int rows;         // its tokens; 0: the slot is unused
};

// By one whole warp: the episode of slot s is the last e with start(e) / 64 +
// e <= s, found by a 32-ary search.  Lanes of the last round hold neighbouring
// episodes' starts, so the episode's range comes along with it.
__device__ __forceinline__ Chunk chunk_of(const int32_t* ends, int32_t episodes, int32_t tokens, int32_t slot) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = episodes;      // the answer lies in [lo, lo + n)
    int32_t start;
    int last;
    while (true) {
        const int step = (n + 31) / 32;
        const int e = lo + lane * step;
        const bool in = lane * step < n;
        start = in && e > 0 ? min(max(ends[e - 1], 0), tokens) : 0;
        const unsigned hits = __ballot_sync(0xffffffffu, in && start / kChunk + e <= slot);
        last = hits ? 31 - __clz(hits) : 0;
        lo += last * step;
        if (step == 1) break;
        n = min(step, n - last * step);
    }
    const int32_t from = __shfl_sync(0xffffffffu, start, last), next = __shfl_sync(0xffffffffu, start, (last + 1) & 31);
    const int32_t end = last + 1 < n ? next : ends[lo];
    const int32_t to = min(max(end, from), tokens);
    const int c = slot - (from / kChunk + lo);
    return {(int64_t)from + c * kChunk, c < 0 ? 0 : min(to - from - c * kChunk, kChunk)};
}

}  // namespace delta
}  // namespace ofrl
