// Per chunk of 64 tokens, independently of every state: the power-of-two
// scaled keys and queries, the decays, P and T = (1 + A)^-1 (see
// delta_mma.cuh for what is left where).
//
// One CTA of four warps per (chunk, key head); the products K K^T and Q K^T
// are made once and serve every value head of the group.
//
// T.  1 + A is unit lower triangular with blocks of 16.  Warp w inverts the
// diagonal block w by forward substitution (a lane per column) and then owns
// T's block column w: transposed, its blocks are mma accumulators of the warp
// and feed the next product as its A operand without leaving registers,
//   T_rw^T = -(sum_{s=w}^{r-1} T_sw^T A_rs^T) T_rr^T.
// Substitution, not a series of powers of A: with correlated keys the powers
// grow before they cancel.  The block products use bf16 planes (two, or three
// where 22 bits are kept): T's elements have no bound known beforehand.

#include "delta_mma.cuh"

namespace ofrl {
namespace delta {
namespace {

constexpr int kPrepThreads = 128;

struct PrepArgs {
    ofrl_delta_shape shape;
    ofrl_delta_tokens in;
    const int32_t* ends;
    int32_t episodes;
    uint8_t* keys;
    uint8_t* pairs;
    int32_t* status;
};

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&x)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack_b(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// Power of two that divides a row: its largest magnitude becomes [1, 2).
__device__ __forceinline__ float row_unit(float amax) {
    const int e = (int)((__float_as_uint(amax) >> 23) & 255u);
    if (e == 255 || amax == 0.0f) return 1.0f;
    return __uint_as_float((uint32_t)min(max(e, 127 - 60), 127 + 60) << 23);
}

// T: token type; DK: padded key width; NM: planes of T and P.
template <typename T, int DK, int NM>
__global__ void __launch_bounds__(kPrepThreads) delta_prep_kernel(const __grid_constant__ PrepArgs a) {
    constexpr int NT = sizeof(T) == 4 ? 2 : 1, CG = DK / 8, KS = DK / 16;
    constexpr int NB = NM + 1;            // bf16 planes inside the inversion
    constexpr int kKey = kChunk * DK * 2;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* kimg = smem;                           // [NT] K^ planes
    uint8_t* qimg = kimg + NT * kKey;               // [NT]
    uint8_t* aimg = qimg + NT * kKey;               // [NB] A's blocks below the diagonal
    uint8_t* timg = aimg + NB * kSquare;            // [NB][4] T's diagonal blocks, 2x2 tiles each
    float* diag = reinterpret_cast<float*>(timg + NB * 4 * 4 * kTile);   // [4][16][17]
    float* vec = diag + 4 * 16 * 17;                // [V_COUNT][64]
    float* kap = vec + V_COUNT * kChunk;            // [64]
    float* kqv = kap + kChunk;                      // [64]
    __shared__ int s_at[3];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hk = a.shape.k_heads, hv = a.shape.v_heads, group = hv / hk, dk = a.shape.k_dim;
    const int64_t slot = blockIdx.x / hk;
    const int khead = blockIdx.x % hk;
    const int32_t tokens = (int32_t)a.in.tokens;
    if (warp == 0) {
        const int e = episode_of(a.ends, a.episodes, tokens, (int32_t)slot);
        const Span sp = span_of(a.ends, e, tokens);
        const int c = (int)slot - (sp.start / kChunk + e);
        if (lane == 0) {
            s_at[0] = sp.start + c * kChunk;
            s_at[1] = c < 0 ? 0 : min(sp.len - c * kChunk, kChunk);
        }
    }
    if (slot == 0 && khead == 0)
        for (int e = threadIdx.x; e < a.episodes; e += kPrepThreads)
            if (span_bad(a.ends, e, tokens)) atomicAdd(a.status + OFRL_STAT_BAD_INDEX, 1);
    __syncthreads();
    const int rows = s_at[1];
    if (rows <= 0) return;
    const int64_t tok = s_at[0];

    // K and Q: a warp takes eight rows at a time, lane = row + 8 * column
    // group, so that a store of 8 lanes fills one 8x8 block.
    uint8_t* keys = a.keys + (slot * hk + khead) * KeyImage::bytes(DK, NT);
    {
        const int r = lane & 7, c4 = lane >> 3;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int rg = warp * 2 + (w & 1);
            const bool isq = w >= 2;
            const int row = rg * 8 + r;
            const T* p = isq ? static_cast<const T*>(a.in.q) + (tok + row) * a.in.q_stride + (int64_t)khead * dk
                             : static_cast<const T*>(a.in.k) + (tok + row) * a.in.k_stride + (int64_t)khead * dk;
            float x[CG / 4][8];
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < CG / 4; ++i) {
                const int col = (c4 + 4 * i) * 8;
                if (row < rows && col < dk)
                    load8<T>(p + col, x[i]);
                else
#pragma unroll
                    for (int z = 0; z < 8; ++z) x[i][z] = 0.0f;
#pragma unroll
                for (int z = 0; z < 8; ++z) m = fmaxf(m, fabsf(x[i][z]));
            }
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
            const float unit = row_unit(m), inv = pow2_inv(unit);
            if (c4 == 0) (isq ? kqv : kap)[row] = unit;
#pragma unroll
            for (int i = 0; i < CG / 4; ++i) {
                uint32_t pl[4][NT];
#pragma unroll
                for (int z = 0; z < 4; ++z) planes_h<NT>(x[i][2 * z] * inv, x[i][2 * z + 1] * inv, pl[z]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint4 v = make_uint4(pl[0][n], pl[1][n], pl[2][n], pl[3][n]);
                    const int at = n * kKey + (rg * CG + c4 + 4 * i) * kTile + r * 16;
                    *reinterpret_cast<uint4*>((isq ? qimg : kimg) + at) = v;
                    *reinterpret_cast<uint4*>(keys + (isq ? NT * kKey : 0) + at) = v;
                }
            }
        }
    }
    __syncthreads();

    // K K^T rows of block `warp`, Q K^T rows of block 3 - warp: five 16x16
    // blocks on or below the diagonal for every warp.
    const int rk = warp, rq = 3 - warp;
    float kk[8][4], qk[8][4];
    zero(kk);
    zero(qk);
    {
        const int m = lane >> 3, r = lane & 7;
        const uint32_t kb = umma::smem_u32(kimg), qb = umma::smem_u32(qimg);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            uint32_t fk[NT][4], fq[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) {   // A operands: row halves (m & 1), k halves (m >> 1)
                const int at = n * kKey + ((2 * rk + (m & 1)) * CG + 2 * k + (m >> 1)) * kTile + r * 16;
                ldsm4(fk[n], kb + at);
                ldsm4(fq[n], qb + at + 2 * (rq - rk) * CG * kTile);
            }
#pragma unroll
            for (int t = 0; t < 8; t += 2)
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    if (t > 2 * rk && t > 2 * rq) continue;
                    uint32_t f[4];
                    ldsm4(f, kb + j * kKey + ((t + (m >> 1)) * CG + 2 * k + (m & 1)) * kTile + r * 16);
#pragma unroll
                    for (int i = 0; i < NT; ++i)
                        if (i + j < NT) {
                            if (t <= 2 * rk) {
                                mma_h(kk[t], fk[i], f[0], f[1]);
                                mma_h(kk[t + 1], fk[i], f[2], f[3]);
                            }
                            if (t <= 2 * rq) {
                                mma_h(qk[t], fq[i], f[0], f[1]);
                                mma_h(qk[t + 1], fq[i], f[2], f[3]);
                            }
                        }
                }
        }
    }

    const int row4 = lane >> 2, col2 = (lane & 3) * 2;
    for (int head = khead * group; head < (khead + 1) * group; ++head) {
        uint8_t* pairs = a.pairs + (slot * hv + head) * kPairBytes;
        if (warp == 0) {
            // running log2 decays in fp64, kept as a pair of floats: a
            // difference of two of them is then exact to fp32
            double g[2];
            float b[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = 2 * lane + i;
                const bool on = t < rows;
                const float gi = on ? to_f(static_cast<const T*>(a.in.g)[(tok + t) * a.in.g_stride + head]) : 0.0f;
                g[i] = (double)fmaxf(gi, kMinLogDecay) * 1.4426950408889634;
                if (isnan(gi)) g[i] = (double)gi;
                b[i] = on ? to_f(static_cast<const T*>(a.in.beta)[(tok + t) * a.in.beta_stride + head]) : 0.0f;
            }
            double sum = g[0] + g[1];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double up = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += up;
            }
            const double total = __shfl_sync(0xffffffffu, sum, 31);
            const double G[2] = {sum - g[1], sum};
            float most = 1.0f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = 2 * lane + i;
                const float hi = (float)G[i];
                vec[V_GHI * kChunk + t] = hi;
                vec[V_GLO * kChunk + t] = (float)(G[i] - (double)hi);
                const float gam = exp2f(hi), rest = exp2f((float)(total - G[i]));
                const float bk = b[i] * kap[t] * kap[t], qs = t < rows ? a.in.scale * kqv[t] : 0.0f;
                vec[V_GAM * kChunk + t] = gam;
                vec[V_REST * kChunk + t] = rest;
                vec[V_BETA * kChunk + t] = bk;
                vec[V_KINV * kChunk + t] = pow2_inv(kap[t]);
                vec[V_QINV * kChunk + t] = pow2_inv(kqv[t]);
                vec[V_QS * kChunk + t] = qs;
                vec[V_OS * kChunk + t] = qs * gam;
                vec[V_DV * kChunk + t] = b[i] * kap[t];
                vec[V_DS * kChunk + t] = bk * gam;
                most = fmaxf(most, rest);
            }
            most = warp_max(most);
            if (lane == 0) vec[V_MISC * kChunk] = most;
        }
        __syncthreads();
        const float *ghi = vec + V_GHI * kChunk, *glo = vec + V_GLO * kChunk, *beta = vec + V_BETA * kChunk;
        auto decay = [&](int i, int j) { return exp2f((ghi[i] - ghi[j]) + (glo[i] - glo[j])); };
        // P to global memory; A's blocks below the diagonal as images, the
        // diagonal block as floats
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            float p[4] = {0, 0, 0, 0};
            if (t <= 2 * rq + 1)
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const int i = rq * 16 + row4 + (z >> 1) * 8, j = t * 8 + col2 + (z & 1);
                    if (j <= i) p[z] = qk[t][z] * decay(i, j) * kPScale;
                }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t pl[NM];
                planes_h<NM>(p[2 * h], p[2 * h + 1], pl);
#pragma unroll
                for (int n = 0; n < NM; ++n)
                    *reinterpret_cast<uint32_t*>(pairs + kSquare + n * kPairFirst + ((2 * rq + h) * 8 + t) * kTile +
                                                 lane * 4) = pl[n];
            }
            if (t < 2 * rk) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x[2];
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const int i = rk * 16 + row4 + h * 8, j = t * 8 + col2 + z;
                        x[z] = beta[i] * kk[t][2 * h + z] * decay(i, j);
                    }
                    uint32_t pl[NB];
                    planes_b<NB>(x[0], x[1], pl);
#pragma unroll
                    for (int n = 0; n < NB; ++n)
                        *reinterpret_cast<uint32_t*>(aimg + n * kSquare + ((2 * rk + h) * 8 + t) * kTile + lane * 4) = pl[n];
                }
            } else if (t <= 2 * rk + 1) {
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const int li = row4 + (z >> 1) * 8, lj = (t - 2 * rk) * 8 + col2 + (z & 1);
                    const int i = rk * 16 + li, j = rk * 16 + lj;
                    diag[(rk * 16 + li) * 17 + lj] = lj < li ? beta[i] * kk[t][z] * decay(i, j) : 0.0f;
                }
            }
        }
        __syncwarp();
        {
            float x[16];
            const float* A = diag + warp * 16 * 17;
            const int c = lane & 15;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float s = i == c ? 1.0f : 0.0f;
#pragma unroll
                for (int j = 0; j < i; ++j) s = fmaf(-A[i * 17 + j], x[j], s);
                x[i] = s;
            }
            __syncwarp();
            if (lane < 16)
#pragma unroll
                for (int i = 0; i < 16; ++i) diag[(warp * 16 + c) * 17 + i] = x[i];   // now T^T: row j, column i
            __syncwarp();
        }
        // own diagonal block, transposed, as accumulator tiles; and as the B
        // operand T_rr [n = i][k = j] for the other warps
        float tb[4][2][4];            // T_rw^T for r = 0 .. 3
        uint32_t tp[3][NB][4];        // its planes as A operands
#pragma unroll
        for (int r = 0; r < 4; ++r) zero(tb[r]);
        const float* D = diag + warp * 16 * 17;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t pl[NB];
                // rows i = row4 + 8 h, columns j = 8 t + col2: element T[i][j] = D[j][i]
                planes_b<NB>(D[(t * 8 + col2) * 17 + row4 + 8 * h], D[(t * 8 + col2 + 1) * 17 + row4 + 8 * h], pl);
#pragma unroll
                for (int n = 0; n < NB; ++n)
                    *reinterpret_cast<uint32_t*>(timg + ((n * 4 + warp) * 4 + h * 2 + t) * kTile + lane * 4) = pl[n];
            }
        __syncthreads();
        {
            const int m = lane >> 3, r8 = lane & 7;
            const uint32_t ab = umma::smem_u32(aimg), tbase = umma::smem_u32(timg);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                if (w != warp) continue;      // w is a constant below: registers are indexed statically
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        tb[w][t][z] = D[(row4 + (z >> 1) * 8) * 17 + t * 8 + col2 + (z & 1)];
#pragma unroll
                for (int r = w + 1; r < 4; ++r) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {      // planes of the block made last
                        uint32_t pl[NB];
                        const float* x = tb[r - 1][i >> 1] + (i & 1) * 2;
                        planes_b<NB>(x[0], x[1], pl);
#pragma unroll
                        for (int n = 0; n < NB; ++n) tp[r - 1][n][i] = pl[n];
                    }
                    float z[2][4];
                    zero(z);
#pragma unroll
                    for (int s = w; s < r; ++s)
#pragma unroll
                        for (int j = 0; j < NB; ++j) {
                            uint32_t f[4];
                            ldsm4(f, ab + j * kSquare + ((2 * r + (m >> 1)) * 8 + 2 * s + (m & 1)) * kTile + r8 * 16);
#pragma unroll
                            for (int i = 0; i < NB; ++i)
                                if (i + j < NB) {
                                    mma_b(z[0], tp[s][i], f[0], f[1]);
                                    mma_b(z[1], tp[s][i], f[2], f[3]);
                                }
                        }
                    uint32_t zp[NB][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t pl[NB];
                        const float* x = z[i >> 1] + (i & 1) * 2;
                        planes_b<NB>(-x[0], -x[1], pl);
#pragma unroll
                        for (int n = 0; n < NB; ++n) zp[n][i] = pl[n];
                    }
#pragma unroll
                    for (int j = 0; j < NB; ++j) {
                        uint32_t f[4];
                        ldsm4(f, tbase + ((j * 4 + r) * 4 + (m >> 1) * 2 + (m & 1)) * kTile + r8 * 16);
#pragma unroll
                        for (int i = 0; i < NB; ++i)
                            if (i + j < NB) {
                                mma_b(tb[r][0], zp[i], f[0], f[1]);
                                mma_b(tb[r][1], zp[i], f[2], f[3]);
                            }
                    }
                }
            }
        }
        // block column of T^T to global memory, with its power of two
        float mx = 0.0f;
#pragma unroll
        for (int r = 0; r < 4; ++r) mx = fmaxf(mx, tile_max(tb[r]));
        const float up = scale_up(mx);
        if (lane < 16) {
            const int j = warp * 16 + lane;
            const float inv = pow2_inv(up);
            vec[V_TINV * kChunk + j] = inv;
            vec[V_XV * kChunk + j] = vec[V_DV * kChunk + j] * inv;
            vec[V_XS * kChunk + j] = vec[V_DS * kChunk + j] * inv;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t pl[NM];
                    planes_h<NM>(tb[r][t][2 * h] * up, tb[r][t][2 * h + 1] * up, pl);
#pragma unroll
                    for (int n = 0; n < NM; ++n)
                        *reinterpret_cast<uint32_t*>(pairs + n * kPairFirst + ((2 * warp + h) * 8 + 2 * r + t) * kTile +
                                                     lane * 4) = pl[n];
                }
        __syncthreads();
        for (int i = threadIdx.x; i < kVecBytes / 16; i += kPrepThreads)
            reinterpret_cast<uint4*>(pairs + 2 * kSquare)[i] = reinterpret_cast<const uint4*>(vec)[i];
        __syncthreads();
    }
}

template <typename T, int DK, int NM>
cudaError_t run(const PrepArgs& p, int64_t grid, cudaStream_t st) {
    constexpr int NT = sizeof(T) == 4 ? 2 : 1, NB = NM + 1;
    constexpr int smem = 2 * NT * kChunk * DK * 2 + NB * kSquare + NB * 16 * kTile + 4 * 16 * 17 * 4 + kVecBytes +
                         2 * kChunk * 4;
    static bool set = false;
    if (!set) {
        const cudaError_t e = cudaFuncSetAttribute(delta_prep_kernel<T, DK, NM>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        set = true;
    }
    delta_prep_kernel<T, DK, NM><<<(unsigned)grid, kPrepThreads, smem, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prep(const SeqLaunch& a, const Prepared& to, int planes, cudaStream_t st) {
    PrepArgs p;
    p.shape = a.shape;
    p.in = a.in;
    p.ends = a.ends;
    p.episodes = a.episodes;
    p.keys = to.keys;
    p.pairs = to.pairs;
    p.status = a.status;
    const int64_t grid = slots_of(a.in.tokens, a.episodes) * a.shape.k_heads;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    const bool wide = a.shape.k_dim > 64;
    if (a.shape.dtype == OFRL_DTYPE_F32) return wide ? run<float, 128, 2>(p, grid, st) : run<float, 64, 2>(p, grid, st);
    if (planes == 2)
        return wide ? run<__nv_bfloat16, 128, 2>(p, grid, st) : run<__nv_bfloat16, 64, 2>(p, grid, st);
    return wide ? run<__nv_bfloat16, 128, 1>(p, grid, st) : run<__nv_bfloat16, 64, 1>(p, grid, st);
}

}  // namespace delta
}  // namespace ofrl
