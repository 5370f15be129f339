// The two passes over an episode's chunks in order: the forward pass that
// carries S and makes the outputs, and the backward pass that carries dS and
// makes dv (see delta_seq.cu for the formulas, delta_mma.cuh for the scaled
// quantities and delta_prep.cu for what is ready before).
//
// Transposed, every product of the recurrence has the value channels as its
// rows, and nothing mixes rows:
//   forward   X^T = v^ - gamma (S K^T),  U^T = (beta X^T) T^T,  O^T = gamma (S Q^T) + U^T P^T,
//             S <- gamma_last S + (rest U^T) K
//   backward  dU^T = dO^T P + rest (dS K^T),  R^T = dU^T T,  dv^ = beta R^T,
//             dS <- gamma_last dS + (gamma dO^T) Q - (gamma dv^T) K
// (columns = tokens; gamma, rest, beta scale columns).  So a warp owns 16
// value channels for the whole episode: S lives in its registers as mma
// accumulators, whose layout is that of the next product's A operand, and
// nothing passes between warps.  One more warp keeps a ring of stages filled
// by bulk copies.  tcgen05 would run these products faster but needs each
// intermediate through TMEM and a CTA-wide hand-over per product, four per
// chunk, for 64-column tiles.

#include "delta_mma.cuh"

namespace ofrl {
namespace delta {
namespace {

constexpr int kWarps = 4;                         // computing warps, 16 value channels each
constexpr int kSlice = kWarps * 16;               // value channels per CTA
constexpr int kChainThreads = (kWarps + 1) * 32;
constexpr uint64_t kWaitNs = 1000000000ull;       // a wait gives up after 1 s

struct ChainArgs {
    ofrl_delta_shape shape;
    ofrl_delta_tokens in;
    const int32_t* ends;
    int32_t episodes;
    const uint8_t* keys;
    const uint8_t* pairs;
    const float* first;      // forward: initial states; backward: gradients of the final ones
    float* last;             // forward: final states; backward: gradients of the initial ones
    void* out;               // forward: outputs; backward: dv
    int64_t out_stride;
    const void* rows;        // forward: v; backward: dout
    int64_t row_stride;
    uint8_t* state_img;      // per (slot, head): S (forward) or dS (backward) before the chunk is taken in, or null
    uint8_t* vec_img;        // per (slot, head): U (forward) or R (backward)
    float* state_unit;       // [slot][head][8]: powers of two of their 16-row blocks
    float* vec_unit;
    int32_t* status;
};

template <typename T>
__host__ __device__ constexpr int row_pitch() { return kSlice * (int)sizeof(T) + 16; }

// One stage: K^ and Q^ planes, T^T / P / vectors (/ second planes), token rows.
template <typename T, int DK, int NM>
struct Stage {
    static constexpr int NT = sizeof(T) == 4 ? 2 : 1;
    static constexpr int kKey = kChunk * DK * 2;
    static constexpr int kKeys = 2 * NT * kKey;
    static constexpr int kPairs = NM == 2 ? (int)kPairBytes : (int)kPairFirst;
    static constexpr int kRows = kChunk * row_pitch<T>();
    static constexpr int kBytes = (kKeys + kPairs + kRows + 127) / 128 * 128;
    static constexpr int kOut = sizeof(T) == 2 ? kWarps * kChunk * 48 : 0;     // staging of bf16 outputs
    // three stages where two CTAs then share an SM, else two where they fit
    static constexpr int kCount = 3 * kBytes <= 100 * 1024 ? 3 : 2 * kBytes + kOut <= 226 * 1024 ? 2 : 1;
    static constexpr int kShared = kCount * kBytes + kOut;
    static_assert(kShared <= 226 * 1024, "shared memory");
};

// Token rows of one chunk, transposed: x[t][z] = row value at (channel row4 +
// (z >> 1) * 8 of the warp, token 8 t + col2 + (z & 1)).
template <typename T>
__device__ __forceinline__ void load_transposed(const uint8_t* rows, float (&x)[8][4], int warp) {
    const int lane = threadIdx.x & 31;
    if constexpr (sizeof(T) == 2) {
        const int m = lane >> 3, r = lane & 7;
#pragma unroll
        for (int t = 0; t < 8; t += 2) {
            uint32_t f[4];   // matrices: (token group t + (m >> 1), channel half m & 1)
            ldsm4t(f, umma::smem_u32(rows) + ((t + (m >> 1)) * 8 + r) * row_pitch<T>() + (warp * 2 + (m & 1)) * 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 v = unpack_b(f[i]);
                x[t + (i >> 1)][(i & 1) * 2] = v.x;
                x[t + (i >> 1)][(i & 1) * 2 + 1] = v.y;
            }
        }
    } else {
        const int row4 = lane >> 2, col2 = (lane & 3) * 2;
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int z = 0; z < 4; ++z)
                x[t][z] = *reinterpret_cast<const float*>(rows + (t * 8 + col2 + (z & 1)) * row_pitch<T>() +
                                                          (warp * 16 + row4 + (z >> 1) * 8) * 4);
    }
}

// The inverse: writes x to rows [64 tokens][16 channels] of global memory
// through the warp's staging area (bf16) or directly (fp32).
template <typename T>
__device__ __forceinline__ void store_transposed(const float (&x)[8][4], T* to, int64_t stride, int rows, int channels,
                                                 uint8_t* stage) {
    const int lane = threadIdx.x & 31;
    if constexpr (sizeof(T) == 2) {
        constexpr int kPitch = 48;      // 16 channels are 32 bytes
        const int m = lane >> 3, r = lane & 7;
        __syncwarp();
#pragma unroll
        for (int t = 0; t < 8; t += 2)
            stsm4t(umma::smem_u32(stage) + ((t + (m >> 1)) * 8 + r) * kPitch + (m & 1) * 16, pack_b(x[t][0], x[t][1]),
                   pack_b(x[t][2], x[t][3]), pack_b(x[t + 1][0], x[t + 1][1]), pack_b(x[t + 1][2], x[t + 1][3]));
        __syncwarp();
        const int half = lane & 1;
        if (half * 8 < channels)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = i * 16 + (lane >> 1);
                if (row < rows)
                    *reinterpret_cast<uint4*>(to + row * stride + half * 8) =
                        *reinterpret_cast<const uint4*>(stage + row * kPitch + half * 16);
            }
    } else {
        const int row4 = lane >> 2, col2 = (lane & 3) * 2;
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const int row = t * 8 + col2 + (z & 1), ch = row4 + (z >> 1) * 8;
                if (row < rows && ch < channels) to[row * stride + ch] = x[t][z];
            }
    }
}

// Fragments of a [16 x 16 KA] accumulator block to the rows rg * 8 .. of an
// image in global memory, cut into slices of 8 * SG columns.
template <int SG, int N, int KA>
__device__ __forceinline__ void store_image(uint8_t* img, int64_t plane, const uint32_t (&a)[N][KA][4], int rg, int RG) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int k = 0; k < KA; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int cg = 2 * k + (i >> 1);
                *reinterpret_cast<uint32_t*>(img + n * plane + ((cg / SG * RG + rg + (i & 1)) * SG + cg % SG) * kTile +
                                             lane * 4) = a[n][k][i];
            }
}

template <int NT>
__device__ __forceinline__ void load_state(const float* from, float (&s)[NT][4], int row0, int dv, int dk) {
    const int lane = threadIdx.x & 31, row4 = lane >> 2, col2 = (lane & 3) * 2;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = row0 + row4 + 8 * h, c = t * 8 + col2;
            float2 v = make_float2(0.0f, 0.0f);
            if (from != nullptr && r < dv && c < dk) v = *reinterpret_cast<const float2*>(from + (int64_t)r * dk + c);
            s[t][2 * h] = v.x;
            s[t][2 * h + 1] = v.y;
        }
}

template <int NT>
__device__ __forceinline__ void store_state(float* to, const float (&s)[NT][4], int row0, int dv, int dk) {
    const int lane = threadIdx.x & 31, row4 = lane >> 2, col2 = (lane & 3) * 2;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = row0 + row4 + 8 * h, c = t * 8 + col2;
            if (r < dv && c < dk)
                *reinterpret_cast<float2*>(to + (int64_t)r * dk + c) = make_float2(s[t][2 * h], s[t][2 * h + 1]);
        }
}

struct Work {
    int e, head, khead, slice;
    Span sp;
    int chunks;
    int64_t slot0;
};
__device__ __forceinline__ Work work_of(const ChainArgs& a) {
    Work w;
    const int hv = a.shape.v_heads, slices = (a.shape.v_dim + kSlice - 1) / kSlice;
    w.slice = blockIdx.x % slices;
    const int64_t item = blockIdx.x / slices;
    w.e = (int)(item / hv);
    w.head = (int)(item % hv);
    w.khead = w.head / (hv / a.shape.k_heads);
    w.sp = span_of(a.ends, w.e, (int32_t)a.in.tokens);
    w.chunks = (w.sp.len + kChunk - 1) / kChunk;
    w.slot0 = w.sp.start / kChunk + w.e;
    return w;
}

// The copying warp: chunks in the order of the pass, one stage each.
template <typename T, int DK, int NM, bool REVERSE>
__device__ __forceinline__ void copy_chunks(const ChainArgs& a, const Work& w, uint8_t* ring, uint64_t* full,
                                            uint64_t* empty, volatile int* dead) {
    using St = Stage<T, DK, NM>;
    const int lane = threadIdx.x & 31;
    const int dv = a.shape.v_dim;
    const int channels = min(kSlice, dv - w.slice * kSlice);
    for (int n = 0; n < w.chunks; ++n) {
        const int st = n % St::kCount;
        const int c = REVERSE ? w.chunks - 1 - n : n;
        bool ok = true;
        if (n >= St::kCount) ok = umma::mbar_wait(&empty[st], (uint32_t)(n / St::kCount - 1) & 1u, kWaitNs);
        if (__any_sync(0xffffffffu, !ok) || *dead) {      // wind down: wait, within limits, for copies in flight
            *dead = 1;
            for (int k = max(n - St::kCount, 0); k < n; ++k)
                umma::mbar_wait(&full[k % St::kCount], (uint32_t)(k / St::kCount) & 1u, kWaitNs);
            return;
        }
        const int rows = min(kChunk, w.sp.len - c * kChunk);
        uint8_t* s = ring + st * St::kBytes;
        const int64_t slot = w.slot0 + c;
        const uint32_t row_bytes = (uint32_t)(channels * sizeof(T));
        if (lane == 0) {
            umma::mbar_expect_tx(&full[st], (uint32_t)(St::kKeys + St::kPairs) + (uint32_t)rows * row_bytes);
            umma::bulk_g2s(s, a.keys + (slot * a.shape.k_heads + w.khead) * KeyImage::bytes(DK, St::NT), St::kKeys,
                           &full[st]);
            umma::bulk_g2s(s + St::kKeys, a.pairs + (slot * a.shape.v_heads + w.head) * kPairBytes, St::kPairs,
                           &full[st]);
        }
        __syncwarp();
        const T* from = static_cast<const T*>(a.rows) + ((int64_t)w.sp.start + c * kChunk) * a.row_stride +
                        (int64_t)w.head * dv + w.slice * kSlice;
        for (int r = lane; r < rows; r += 32)
            umma::bulk_g2s(s + St::kKeys + St::kPairs + r * row_pitch<T>(), from + r * a.row_stride, row_bytes, &full[st]);
    }
}

// Wait of a computing warp for stage st; false: give up.
__device__ __forceinline__ bool stage_ready(uint64_t* full, int st, int turn, volatile int* dead) {
    const bool ok = umma::mbar_wait(&full[st], (uint32_t)turn & 1u, kWaitNs);
    if (__any_sync(0xffffffffu, !ok)) *dead = 1;
    return __all_sync(0xffffffffu, ok);
}

// NM: planes of S, X, U (and of T and P).  SAVE: S and U go to images for the
// backward pass (NS planes).
template <typename T, int DK, int NM, bool SAVE>
__global__ void __launch_bounds__(kChainThreads) delta_forward_kernel(const __grid_constant__ ChainArgs a) {
    using St = Stage<T, DK, NM>;
    constexpr int NT = St::NT, CG = DK / 8, KS = DK / 16;
    constexpr int NO = sizeof(T) == 4 ? 2 : 1;      // planes of the operands that only the outputs see
    constexpr int NS = NT;                          // planes of the saved images
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t full[3], empty[3];
    __shared__ int dead;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Work w = work_of(a);
    if (threadIdx.x == 0) {
        for (int i = 0; i < 3; ++i) {
            umma::mbar_init(&full[i], 1);
            umma::mbar_init(&empty[i], kWarps);
        }
        dead = 0;
        umma::fence_mbar_init();
    }
    __syncthreads();
    if (warp == kWarps) {
        copy_chunks<T, DK, NM, false>(a, w, smem, full, empty, &dead);
    } else {
        const int dk = a.shape.k_dim, dv = a.shape.v_dim, hv = a.shape.v_heads;
        const int row0 = w.slice * kSlice + warp * 16;
        const int row4 = lane >> 2, col2 = (lane & 3) * 2;
        const int64_t states = ((int64_t)w.e * hv + w.head) * dv * dk;
        float S[DK / 8][4];
        load_state(a.first ? a.first + states : nullptr, S, row0, dv, dk);
        for (int c = 0; c < w.chunks; ++c) {
            const int st = c % St::kCount;
            if (!stage_ready(full, st, c / St::kCount, &dead)) break;
            const uint8_t* s = smem + st * St::kBytes;
            const uint32_t kimg = umma::smem_u32(s), qimg = kimg + NT * St::kKey, pair = kimg + St::kKeys;
            const float* vec = reinterpret_cast<const float*>(s + St::kKeys + 2 * kSquare);
            const int rows = min(kChunk, w.sp.len - c * kChunk);
            if (row0 < dv) {
                const int64_t at = (w.slot0 + c) * hv + w.head;
                float X[8][4], O[8][4];
                zero(X);
                zero(O);
                const float s_up = scale_up(tile_max(S)), s_inv = pow2_inv(s_up);
                {
                    uint32_t f[NM][KS][4];
                    to_frags<NM>(S, s_up, f);
                    gemm<KS, 8, NM, NT, false>(X, f, kimg, St::kKey, CG, 0);
                    if constexpr (NO == NM) {
                        gemm<KS, 8, NM, NT, false>(O, f, qimg, St::kKey, CG, 0);
                    } else {
                        uint32_t f0[1][KS][4];
#pragma unroll
                        for (int k = 0; k < KS; ++k)
#pragma unroll
                            for (int i = 0; i < 4; ++i) f0[0][k][i] = f[0][k][i];
                        gemm<KS, 8, 1, NT, false>(O, f0, qimg, St::kKey, CG, 0);
                    }
                    if constexpr (SAVE) {
                        uint32_t g[NS][KS][4];
#pragma unroll
                        for (int n = 0; n < NS; ++n)
#pragma unroll
                            for (int k = 0; k < KS; ++k)
#pragma unroll
                                for (int i = 0; i < 4; ++i) g[n][k][i] = f[n][k][i];
                        const int dvp = pad_dim(dv);
                        store_image<NT == 1 ? CG : kSliceCols / 8>(a.state_img + at * NS * dvp * DK * 2, (int64_t)dvp * DK * 2, g, row0 / 8,
                                                    dvp / 8);
                        if (lane == 0) a.state_unit[at * 8 + row0 / 16] = s_inv;
                    }
                }
                {
                    float V[8][4];
                    load_transposed<T>(s + St::kKeys + St::kPairs, V, warp);
#pragma unroll
                    for (int t = 0; t < 8; ++t)
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            const int i = t * 8 + col2 + z;
                            const float gam = vec[V_GAM * kChunk + i] * s_inv, kinv = vec[V_KINV * kChunk + i];
                            const float y = vec[V_BETA * kChunk + i] * vec[V_TINV * kChunk + i];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const bool on = i < rows && row0 + row4 + 8 * h < dv;   // else never copied
                                X[t][2 * h + z] = on ? y * (V[t][2 * h + z] * kinv - gam * X[t][2 * h + z]) : 0.0f;
                            }
                        }
                }
                float U[8][4];
                zero(U);
                {
                    const float up = scale_up(tile_max(X)), inv = pow2_inv(up);
                    uint32_t f[NM][4][4];
                    to_frags<NM>(X, up, f);
                    gemm<4, 8, NM, NM, true>(U, f, pair, (int)kPairFirst, 8, 0);
#pragma unroll
                    for (int t = 0; t < 8; ++t)
#pragma unroll
                        for (int z = 0; z < 4; ++z) U[t][z] *= inv;
                }
                // X now holds rest U, what the state takes in
#pragma unroll
                for (int t = 0; t < 8; ++t)
#pragma unroll
                    for (int z = 0; z < 4; ++z) X[t][z] = U[t][z] * vec[V_REST * kChunk + t * 8 + col2 + (z & 1)];
                const float up = scale_up(fmaxf(tile_max(U), tile_max(X))), inv = pow2_inv(up);
                {
                    uint32_t f[NO][4][4];
                    to_frags<NO>(U, up, f);
                    zero(U);
                    gemm<4, 8, NO, NO, false>(U, f, pair + kSquare, (int)kPairFirst, 8, 0);
                    if constexpr (SAVE) {
                        const int dvp = pad_dim(dv);
                        store_image<8>(a.vec_img + at * NS * dvp * kChunk * 2, (int64_t)dvp * kChunk * 2, f, row0 / 8, dvp / 8);
                        if (lane == 0) a.vec_unit[at * 8 + row0 / 16] = inv;
                    }
                }
                const float p_inv = inv * (1.0f / kPScale);
#pragma unroll
                for (int t = 0; t < 8; ++t)
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const int i = t * 8 + col2 + (z & 1);
                        O[t][z] = vec[V_QS * kChunk + i] * (vec[V_GAM * kChunk + i] * s_inv * O[t][z] + p_inv * U[t][z]);
                    }
                {
                    uint32_t f[NM][4][4];
                    to_frags<NM>(X, up, f);
                    const float keep = vec[V_GAM * kChunk + kChunk - 1];
#pragma unroll
                    for (int t = 0; t < DK / 8; t += 4) {
                        float d[4][4];
                        zero(d);
                        gemm<4, 4, NM, NT, true>(d, f, kimg, St::kKey, CG, t);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int z = 0; z < 4; ++z) S[t + i][z] = keep * S[t + i][z] + inv * d[i][z];
                    }
                }
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(&empty[st]);
                store_transposed<T>(O, static_cast<T*>(a.out) + ((int64_t)w.sp.start + c * kChunk) * a.out_stride +
                                           (int64_t)w.head * dv + row0,
                                    a.out_stride, rows, dv - row0, smem + St::kCount * St::kBytes + warp * kChunk * 48);
            } else if (lane == 0) {
                umma::mbar_arrive(&empty[st]);
            }
        }
        if (a.last) store_state(a.last + states, S, row0, dv, dk);
    }
    __syncthreads();
    if (threadIdx.x == 0 && dead) atomicAdd(a.status + OFRL_STAT_TIMEOUT, 1);
}

template <typename T, int DK, int NM>
__global__ void __launch_bounds__(kChainThreads) delta_reverse_kernel(const __grid_constant__ ChainArgs a) {
    using St = Stage<T, DK, NM>;
    constexpr int NT = St::NT, CG = DK / 8, KS = DK / 16, NS = NT;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t full[3], empty[3];
    __shared__ int dead;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Work w = work_of(a);
    if (threadIdx.x == 0) {
        for (int i = 0; i < 3; ++i) {
            umma::mbar_init(&full[i], 1);
            umma::mbar_init(&empty[i], kWarps);
        }
        dead = 0;
        umma::fence_mbar_init();
    }
    __syncthreads();
    if (warp == kWarps) {
        copy_chunks<T, DK, NM, true>(a, w, smem, full, empty, &dead);
    } else {
        const int dk = a.shape.k_dim, dv = a.shape.v_dim, hv = a.shape.v_heads;
        const int row0 = w.slice * kSlice + warp * 16;
        const int row4 = lane >> 2, col2 = (lane & 3) * 2;
        const int dvp = pad_dim(dv);
        const int64_t states = ((int64_t)w.e * hv + w.head) * dv * dk;
        float S[DK / 8][4];
        load_state(a.first ? a.first + states : nullptr, S, row0, dv, dk);
        for (int n = 0; n < w.chunks; ++n) {
            const int st = n % St::kCount, c = w.chunks - 1 - n;
            if (!stage_ready(full, st, n / St::kCount, &dead)) break;
            const uint8_t* s = smem + st * St::kBytes;
            const uint32_t kimg = umma::smem_u32(s), qimg = kimg + NT * St::kKey, pair = kimg + St::kKeys;
            const float* vec = reinterpret_cast<const float*>(s + St::kKeys + 2 * kSquare);
            const int rows = min(kChunk, w.sp.len - c * kChunk);
            if (row0 < dv) {
                const int64_t at = (w.slot0 + c) * hv + w.head;
                float U[8][4];
                zero(U);
                const float s_up = scale_up(tile_max(S)), s_inv = pow2_inv(s_up);
                {
                    uint32_t f[NM][KS][4];
                    to_frags<NM>(S, s_up, f);
                    gemm<KS, 8, NM, NT, false>(U, f, kimg, St::kKey, CG, 0);
                    store_image<NT == 1 ? CG : kSliceCols / 8>(a.state_img + at * NS * dvp * DK * 2, (int64_t)dvp * DK * 2, f, row0 / 8,
                                                dvp / 8);
                    if (lane == 0) a.state_unit[at * 8 + row0 / 16] = s_inv;
                }
                float dO[8][4];       // dout scale kq
                load_transposed<T>(s + St::kKeys + St::kPairs, dO, warp);
#pragma unroll
                for (int t = 0; t < 8; ++t)
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const int i = t * 8 + col2 + (z & 1);
                        const bool on = i < rows && row0 + row4 + (z >> 1) * 8 < dv;
                        dO[t][z] = on ? dO[t][z] * vec[V_QS * kChunk + i] : 0.0f;
                        U[t][z] *= vec[V_REST * kChunk + i] * s_inv;
                    }
                {
                    const float up = scale_up(tile_max(dO)), inv = pow2_inv(up) * (1.0f / kPScale);
                    uint32_t f[NM][4][4];
                    to_frags<NM>(dO, up, f);
                    float d[8][4];
                    zero(d);
                    gemm<4, 8, NM, NM, true>(d, f, pair + kSquare, (int)kPairFirst, 8, 0);
#pragma unroll
                    for (int t = 0; t < 8; ++t)
#pragma unroll
                        for (int z = 0; z < 4; ++z) U[t][z] += inv * d[t][z];
                }
                float R[8][4];
                zero(R);
                {
                    const float up = scale_up(tile_max(U)), inv = pow2_inv(up);
                    uint32_t f[NM][4][4];
                    to_frags<NM>(U, up, f);
                    gemm<4, 8, NM, NM, false>(R, f, pair, (int)kPairFirst, 8, 0);
#pragma unroll
                    for (int t = 0; t < 8; ++t)
#pragma unroll
                        for (int z = 0; z < 4; ++z) R[t][z] *= inv * vec[V_TINV * kChunk + t * 8 + col2 + (z & 1)];
                }
                {
                    const float up = scale_up(tile_max(R));
                    uint32_t f[NS][4][4];
                    to_frags<NS>(R, up, f);
                    store_image<8>(a.vec_img + at * NS * dvp * kChunk * 2, (int64_t)dvp * kChunk * 2, f, row0 / 8, dvp / 8);
                    if (lane == 0) a.vec_unit[at * 8 + row0 / 16] = pow2_inv(up);
                }
                // dv^ in R; gamma dO and gamma dv^ for the state
#pragma unroll
                for (int t = 0; t < 8; ++t)
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const int i = t * 8 + col2 + (z & 1);
                        const float gam = vec[V_GAM * kChunk + i];
                        R[t][z] *= vec[V_BETA * kChunk + i];
                        dO[t][z] *= gam;
                        U[t][z] = -gam * R[t][z];
                        R[t][z] *= vec[V_KINV * kChunk + i];
                    }
                {
                    const float up = scale_up(fmaxf(tile_max(dO), tile_max(U))), inv = pow2_inv(up);
                    uint32_t f[NM][4][4], g[NM][4][4];
                    to_frags<NM>(dO, up, f);
                    to_frags<NM>(U, up, g);
                    const float keep = vec[V_GAM * kChunk + kChunk - 1];
#pragma unroll
                    for (int t = 0; t < DK / 8; t += 4) {
                        float d[4][4];
                        zero(d);
                        gemm<4, 4, NM, NT, true>(d, f, qimg, St::kKey, CG, t);
                        gemm<4, 4, NM, NT, true>(d, g, kimg, St::kKey, CG, t);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int z = 0; z < 4; ++z) S[t + i][z] = keep * S[t + i][z] + inv * d[i][z];
                    }
                }
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(&empty[st]);
                store_transposed<T>(R, static_cast<T*>(a.out) + ((int64_t)w.sp.start + c * kChunk) * a.out_stride +
                                           (int64_t)w.head * dv + row0,
                                    a.out_stride, rows, dv - row0, smem + St::kCount * St::kBytes + warp * kChunk * 48);
            } else if (lane == 0) {
                umma::mbar_arrive(&empty[st]);
            }
        }
        if (a.last) store_state(a.last + states, S, row0, dv, dk);
    }
    __syncthreads();
    if (threadIdx.x == 0 && dead) atomicAdd(a.status + OFRL_STAT_TIMEOUT, 1);
}

template <typename K>
cudaError_t go(K kernel, int smem, const ChainArgs& c, cudaStream_t st) {
    const int slices = (c.shape.v_dim + kSlice - 1) / kSlice;
    const int64_t grid = (int64_t)c.episodes * c.shape.v_heads * slices;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = set_max_shared_carveout(kernel);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)grid, kChainThreads, smem, st>>>(c);
    return cudaGetLastError();
}

template <typename T, int DK, int NM>
cudaError_t forward(const ChainArgs& c, cudaStream_t st) {
    return c.state_img ? go(delta_forward_kernel<T, DK, NM, true>, Stage<T, DK, NM>::kShared, c, st)
                       : go(delta_forward_kernel<T, DK, NM, false>, Stage<T, DK, NM>::kShared, c, st);
}
template <typename T, int DK, int NM>
cudaError_t reverse(const ChainArgs& c, cudaStream_t st) {
    return go(delta_reverse_kernel<T, DK, NM>, Stage<T, DK, NM>::kShared, c, st);
}

ChainArgs base_args(const SeqLaunch& a, const Prepared& p, const Images& img) {
    ChainArgs c;
    c.shape = a.shape;
    c.in = a.in;
    c.ends = a.ends;
    c.episodes = a.episodes;
    c.keys = p.keys;
    c.pairs = p.pairs;
    c.state_img = img.state;
    c.vec_img = img.vec;
    c.state_unit = img.state_unit;
    c.vec_unit = img.vec_unit;
    c.status = a.status;
    return c;
}

}  // namespace

cudaError_t launch_chain_forward(const SeqLaunch& a, const Prepared& p, const Images& img, int planes, cudaStream_t st) {
    ChainArgs c = base_args(a, p, img);
    c.first = a.init;
    c.last = a.final_state;
    c.out = a.out;
    c.out_stride = (int64_t)a.shape.v_heads * a.shape.v_dim;
    c.rows = a.in.v;
    c.row_stride = a.in.v_stride;
    const bool wide = a.shape.k_dim > 64;
    if (a.shape.dtype == OFRL_DTYPE_F32) return wide ? forward<float, 128, 2>(c, st) : forward<float, 64, 2>(c, st);
    if (planes == 2) return wide ? forward<__nv_bfloat16, 128, 2>(c, st) : forward<__nv_bfloat16, 64, 2>(c, st);
    return wide ? forward<__nv_bfloat16, 128, 1>(c, st) : forward<__nv_bfloat16, 64, 1>(c, st);
}

cudaError_t launch_chain_reverse(const SeqLaunch& a, const Prepared& p, const Images& img, cudaStream_t st) {
    ChainArgs c = base_args(a, p, img);
    c.first = a.d_final;
    c.last = a.d_init;
    c.out = a.grads.dv;
    c.out_stride = a.grads.v_stride;
    c.rows = a.dout;
    c.row_stride = (int64_t)a.shape.v_heads * a.shape.v_dim;
    const bool wide = a.shape.k_dim > 64;
    if (a.shape.dtype == OFRL_DTYPE_F32) return wide ? reverse<float, 128, 2>(c, st) : reverse<float, 64, 2>(c, st);
    return wide ? reverse<__nv_bfloat16, 128, 1>(c, st) : reverse<__nv_bfloat16, 64, 1>(c, st);
}

}  // namespace delta
}  // namespace ofrl
