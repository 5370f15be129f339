// Gradients of q, k, log decay and write strength for fp32 tokens, chunk by
// chunk: everything that contracts over the value channels (see delta_seq.cu
// for the formulas and delta_mma.cuh for the scaled quantities).  One CTA of
// eight warps per (chunk, key head), looping over the group's value heads, whose
// gradients it adds up in registers; warp (rb, hf) has the token rows 16 rb ..
// and, of each product's columns, half hf.
//
// Per value head, with N1 = dO U^T and N2 = R U^T:
//   dPD_ij = D_ij N1_ij (j <= i),  E_ij = -D_ij N2_ij (j < i),  M_ij = beta_i E_ij
//   dq_i = gamma_i dO_i S_0 + sum_j dPD_ij k_j
//   dk_i = -gamma_i beta_i R_i S_0 + sum_j M_ij k_j + sum_m dPD_mi q_m + sum_m M_mi k_m + rest_i U_i dS_1
//   dbeta_i = R_i v_i - gamma_i k_i (R_i S_0) + sum_j E_ij (k_i k_j)
//   N_ij = dPD_ij (q_i k_j) + M_ij (k_i k_j)
// (k, v, beta, U, dO scaled as in delta_mma.cuh, dO with scale and kq in it).
// The states come in slices of 32 key channels.
//
// mma.sync with two planes, three products for each one: bound by them and by
// the operands' reads from shared memory.  640 CTAs of 64 x 64 (16384 tokens)
// 61 us.

#include "delta_mma.cuh"

namespace ofrl {
namespace delta {
namespace {

constexpr int kGradThreads = 256;
constexpr uint64_t kWaitNs = 1000000000ull;

struct GradArgs {
    ofrl_delta_shape shape;
    ofrl_delta_tokens in;
    const int32_t* ends;
    int32_t episodes;
    const uint8_t* keys;
    const uint8_t* pairs;
    const uint8_t *s_img, *u_img, *d_img, *r_img;       // S_0, U^T, dS_1, R^T
    const float *s_unit, *u_unit, *d_unit, *r_unit;
    const void* dout;
    ofrl_delta_grads grads;
    int32_t* status;
};

__device__ __forceinline__ int exponent(float pow2) { return (int)((__float_as_uint(pow2) >> 23) & 255u) - 127; }
__device__ __forceinline__ float pow2f(int e) {
    return __uint_as_float((uint32_t)(min(max(e, -126), 127) + 127) << 23);
}
// x 2^e for |e| <= 252.
__device__ __forceinline__ float times_pow2(float x, int e) { return x * pow2f(e / 2) * pow2f(e - e / 2); }
template <int DK, int DV>
struct GradShared {
    static constexpr int NT = 2;                             // planes of the images
    static constexpr int kKey = kChunk * DK * 2;
    static constexpr int kVec = DV * kChunk * 2;             // one plane of U^T or R^T
    static constexpr int kSl = DV * kSliceCols * 2;          // one plane of a state's slice
    static constexpr int kRing = DK == 128 && DV == 128 ? 1 : 2;
    static constexpr int off_u = 2 * NT * kKey;
    static constexpr int off_r = off_u + NT * kVec;
    static constexpr int off_ring = off_r + NT * kVec;
    static constexpr int off_pd = off_ring + kRing * 2 * NT * kSl;
    static constexpr int off_m = off_pd + NT * kSquare;
    static constexpr int off_vec = off_m + NT * kSquare;
    static constexpr int off_sum = off_vec + kVecBytes;
    static constexpr int kSums = (2 * 6 * kChunk + 4 * kChunk + 32 + 32) * 4;
    static constexpr int kBytes = off_sum + kSums;
};

template <int DK, int DV>
__global__ void __launch_bounds__(kGradThreads) delta_grad_kernel(const __grid_constant__ GradArgs a) {
    using Sh = GradShared<DK, DV>;
    constexpr int NT = Sh::NT, CG = DK / 8, KS = DK / 16, KV = DV / 16, SL = DK / kSliceCols, SG = kSliceCols / 8;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bar_keys, bar_head, bar_slice[2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rb = warp & 3, hf = warp >> 2;
    const int m8 = lane >> 3, r8 = lane & 7, row4 = lane >> 2, col2 = (lane & 3) * 2;
    const int hk = a.shape.k_heads, hv = a.shape.v_heads, group = hv / hk, dk = a.shape.k_dim, dv = a.shape.v_dim;
    const int64_t slot = blockIdx.x / hk;
    const int khead = blockIdx.x % hk;
    __shared__ int s_at[3];
    if (warp == 0) {
        const Chunk c = chunk_of(a.ends, a.episodes, (int32_t)a.in.tokens, (int32_t)slot);
        if (lane == 0) {
            s_at[0] = (int)c.tok;
            s_at[1] = c.rows;
            s_at[2] = 0;
            umma::mbar_init(&bar_keys, 1);
            umma::mbar_init(&bar_head, 1);
            umma::mbar_init(&bar_slice[0], 1);
            umma::mbar_init(&bar_slice[1], 1);
            umma::fence_mbar_init();
        }
    }
    pdl_wait();      // what the backward chain leaves
    __syncthreads();
    const int rows = s_at[1];
    if (rows <= 0) return;
    const int64_t tok = s_at[0];
    const int blocks = (dv + 15) / 16;

    uint8_t *kimg = smem, *qimg = smem + NT * Sh::kKey, *uimg = smem + Sh::off_u, *rimg = smem + Sh::off_r;
    uint8_t *ring = smem + Sh::off_ring, *pdimg = smem + Sh::off_pd, *mimg = smem + Sh::off_m;
    const uint32_t kadr = umma::smem_u32(kimg), qadr = umma::smem_u32(qimg), uadr = umma::smem_u32(uimg),
                   radr = umma::smem_u32(rimg), pdadr = umma::smem_u32(pdimg), madr = umma::smem_u32(mimg);
    float* vec = reinterpret_cast<float*>(smem + Sh::off_vec);
    float* sums = reinterpret_cast<float*>(smem + Sh::off_sum);       // [2][6][64] row sums by half
    float* colsum = sums + 2 * 6 * kChunk;                            // [4][64]
    float* wmax = colsum + 4 * kChunk;                                // [8][2]
    float* wsum = wmax + 32;                                          // [8]
    enum { R_N, R_BETA, R_Q, R_K, R_COL, R_RV };

    const int64_t at0 = slot * hv;
    auto copy_slice = [&](int head, int n) {      // thread 0: slice n of S_0 and dS_1
        const int64_t img = (at0 + head) * NT * DV * DK * 2 + (int64_t)n * Sh::kSl;
        uint8_t* to = ring + (n % Sh::kRing) * 2 * NT * Sh::kSl;
        uint64_t* bar = &bar_slice[n % Sh::kRing];
        umma::mbar_expect_tx(bar, 2 * NT * Sh::kSl);
#pragma unroll
        for (int p = 0; p < NT; ++p) {
            umma::bulk_g2s(to + p * Sh::kSl, a.s_img + img + (int64_t)p * DV * DK * 2, Sh::kSl, bar);
            umma::bulk_g2s(to + (NT + p) * Sh::kSl, a.d_img + img + (int64_t)p * DV * DK * 2, Sh::kSl, bar);
        }
    };
    auto copy_head = [&](int head) {
        umma::mbar_expect_tx(&bar_head, 2 * NT * Sh::kVec + kVecBytes);
        umma::bulk_g2s(uimg, a.u_img + (at0 + head) * NT * Sh::kVec, NT * Sh::kVec, &bar_head);
        umma::bulk_g2s(rimg, a.r_img + (at0 + head) * NT * Sh::kVec, NT * Sh::kVec, &bar_head);
        umma::bulk_g2s(vec, a.pairs + (at0 + head) * kPairBytes + 2 * kSquare, kVecBytes, &bar_head);
    };
    if (threadIdx.x == 0) {
        umma::mbar_expect_tx(&bar_keys, 2 * NT * Sh::kKey);
        umma::bulk_g2s(kimg, a.keys + (slot * hk + khead) * KeyImage::bytes(DK, NT), 2 * NT * Sh::kKey, &bar_keys);
        copy_head(khead * group);
        for (int n = 0; n < Sh::kRing && n < SL; ++n) copy_slice(khead * group, n);
    }
    // dO rows i0, i0 + 8 of this thread, as they are; the first head's come while
    // the keys do, where registers allow
    float x[2 * KV][4];
    auto load_dout = [&](int head) {
        const float* po = static_cast<const float*>(a.dout) + (tok * hv + head) * dv;
#pragma unroll
        for (int t = 0; t < 2 * KV; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = rb * 16 + row4 + 8 * h, c = t * 8 + col2;
                float2 v = make_float2(0.0f, 0.0f);
                if (i < rows && c < dv) v = *reinterpret_cast<const float2*>(po + (int64_t)i * hv * dv + c);
                x[t][2 * h] = v.x;
                x[t][2 * h + 1] = v.y;
            }
    };
    constexpr bool kEarly = KV <= 4;
    if (kEarly) load_dout(khead * group);
    bool ok = true;      // a wait that gave up: computing goes on with what is there, nothing is written
    ok &= umma::mbar_wait(&bar_keys, 0, kWaitNs);

    // k k^T and q k^T: rows rb, column tiles 4 hf .. 4 hf + 3
    float kk[4][4], qk[4][4];
    zero(kk);
    zero(qk);
#pragma unroll
    for (int k = 0; k < KS; ++k) {
        uint32_t fk[NT][1][4], fq[NT][1][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int at = n * Sh::kKey + ((2 * rb + (m8 & 1)) * CG + 2 * k + (m8 >> 1)) * kTile + r8 * 16;
            ldsm4(fk[n][0], kadr + at);
            ldsm4(fq[n][0], qadr + at);
        }
        gemm<1, 4, NT, NT, false>(kk, fk, kadr + 2 * k * kTile, Sh::kKey, CG, 4 * hf);
        gemm<1, 4, NT, NT, false>(qk, fq, kadr + 2 * k * kTile, Sh::kKey, CG, 4 * hf);
    }

    float dq[SL][2][4], dkk[SL][2][4];
#pragma unroll
    for (int n = 0; n < SL; ++n) {
        zero(dq[n]);
        zero(dkk[n]);
    }
    uint32_t slice_turn = 0;     // slices taken so far, over all heads
    for (int g = 0; g < group; ++g) {
        const int head = khead * group + g;
        const float su = a.s_unit[at0 + head], uu = a.u_unit[at0 + head], du = a.d_unit[at0 + head],
                    ru = a.r_unit[at0 + head];
        if (!kEarly || g > 0) load_dout(head);
        ok &= umma::mbar_wait(&bar_head, (uint32_t)g & 1u, kWaitNs);
        const float *gam = vec + V_GAM * kChunk, *rest = vec + V_REST * kChunk, *beta = vec + V_BETA * kChunk;
        const float *ghi = vec + V_GHI * kChunk, *glo = vec + V_GLO * kChunk;
        const int i0 = rb * 16 + row4;          // this thread's rows: i0 and i0 + 8

        // dO rows as A operands, times scale and kq, and R v^
        uint32_t fo[NT][KV][4];
        int o_exp;
        float rv[2] = {0.0f, 0.0f};
        {
            const float* pv = static_cast<const float*>(a.in.v) + tok * a.in.v_stride + (int64_t)head * dv;
#pragma unroll
            for (int t = 0; t < 2 * KV; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float f = vec[V_QS * kChunk + i0 + 8 * h];
                    x[t][2 * h] *= f;
                    x[t][2 * h + 1] *= f;
                }
            const float up = scale_up(tile_max(x));
            o_exp = -exponent(up);
            to_frags<NT>(x, up, fo);
            if (hf == 0) {
#pragma unroll
                for (int k = 0; k < KV; ++k) {
                    if (k >= blocks) continue;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        uint32_t f[4];
                        ldsm4t(f, radr + n * Sh::kVec + ((2 * k + (m8 >> 1)) * 8 + 2 * rb + (m8 & 1)) * kTile + r8 * 16);
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const int i = i0 + 8 * (z & 1), c = k * 16 + 8 * (z >> 1) + col2;
                            if (i < rows && c < dv) {
                                const float2 r = unpack_h(f[z]);
                                const float* p = pv + i * a.in.v_stride + c;
                                rv[z & 1] += (r.x * p[0] + r.y * p[1]) * ru;
                            }
                        }
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) rv[h] *= vec[V_KINV * kChunk + i0 + 8 * h];
            }
        }
        // N1 = dO U^T, N2 = R U^T
        float n1[4][4], n2[4][4];
        zero(n1);
        zero(n2);
        const int n1_exp = exponent(uu) + o_exp, n2_exp = exponent(uu) + exponent(ru);
#pragma unroll
        for (int k = 0; k < KV; ++k) {
            if (k >= blocks) continue;
            uint32_t f1[NT][1][4], f2[NT][1][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                ldsm4t(f2[n][0], radr + n * Sh::kVec + ((2 * k + (m8 >> 1)) * 8 + 2 * rb + (m8 & 1)) * kTile + r8 * 16);
#pragma unroll
                for (int z = 0; z < 4; ++z) f1[n][0][z] = fo[n][k][z];
            }
            const uint32_t b = uadr + 2 * k * 8 * kTile;
            gemm<1, 4, NT, NT, true>(n1, f1, b, Sh::kVec, 8, 4 * hf);
            gemm<1, 4, NT, NT, true>(n2, f2, b, Sh::kVec, 8, 4 * hf);
        }
        // dPD in n1, M in n2; row and column sums of N; the beta sum
        float rn[2] = {0.0f, 0.0f}, rbeta[2] = {0.0f, 0.0f};
        float cn[4][2];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            cn[t][0] = cn[t][1] = 0.0f;
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const int h = z >> 1, i = i0 + 8 * h, j = (4 * hf + t) * 8 + col2 + (z & 1);
                const float d = j <= i ? exp2f((ghi[i] - ghi[j]) + (glo[i] - glo[j])) : 0.0f;
                const float pd = j <= i ? times_pow2(n1[t][z], n1_exp) * d : 0.0f;
                const float e = j < i ? -times_pow2(n2[t][z], n2_exp) * d : 0.0f;
                const float mm = beta[i] * e;
                const float x = pd * qk[t][z] + mm * kk[t][z];
                rn[h] += x;
                cn[t][z & 1] += x;
                rbeta[h] += e * kk[t][z];
                n1[t][z] = pd;
                n2[t][z] = mm;
            }
        }
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) cn[t][z] += __shfl_xor_sync(0xffffffffu, cn[t][z], o);
                if (lane < 4) colsum[rb * kChunk + (4 * hf + t) * 8 + col2 + z] = cn[t][z];
            }
        {
            const float m1 = tile_max(n1), m2 = tile_max(n2);
            if (lane == 0) {
                wmax[warp * 2] = m1;
                wmax[warp * 2 + 1] = m2;
            }
        }
        __syncthreads();
        float m1 = 0.0f, m2 = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            m1 = fmaxf(m1, wmax[2 * i]);
            m2 = fmaxf(m2, wmax[2 * i + 1]);
        }
        const float pd_up = scale_up(m1), pd_inv = pow2_inv(pd_up), m_up = scale_up(m2), m_inv = pow2_inv(m_up);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t p1[NT], p2[NT];
                planes_h<NT>(n1[t][2 * h] * pd_up, n1[t][2 * h + 1] * pd_up, p1);
                planes_h<NT>(n2[t][2 * h] * m_up, n2[t][2 * h + 1] * m_up, p2);
                const int at = ((2 * rb + h) * 8 + 4 * hf + t) * kTile + lane * 4;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    *reinterpret_cast<uint32_t*>(pdimg + n * kSquare + at) = p1[n];
                    *reinterpret_cast<uint32_t*>(mimg + n * kSquare + at) = p2[n];
                }
            }
        __syncthreads();

        const int q_exp = exponent(su) + o_exp, k_exp = exponent(su) + exponent(ru), c_exp = exponent(du) + exponent(uu);
        float dotq[2] = {0, 0}, dotk[2] = {0, 0}, dotc[2] = {0, 0}, ss = 0.0f;
#pragma unroll
        for (int n = 0; n < SL; ++n) {
            const int st = n % Sh::kRing;
            ok &= umma::mbar_wait(&bar_slice[st], (slice_turn / Sh::kRing) & 1u, kWaitNs);
            ++slice_turn;
            const uint32_t sadr = umma::smem_u32(ring) + st * 2 * NT * Sh::kSl, dadr = sadr + NT * Sh::kSl;
            float sq[2][4], sk[2][4], sc[2][4];
            zero(sq);
            zero(sk);
            zero(sc);
#pragma unroll
            for (int k = 0; k < KV; ++k) {
                if (k >= blocks) continue;
                uint32_t f1[NT][1][4], f2[NT][1][4], f3[NT][1][4];
#pragma unroll
                for (int p = 0; p < NT; ++p) {
                    const uint32_t at = p * Sh::kVec + ((2 * k + (m8 >> 1)) * 8 + 2 * rb + (m8 & 1)) * kTile + r8 * 16;
                    ldsm4t(f2[p][0], radr + at);
                    ldsm4t(f3[p][0], uadr + at);
#pragma unroll
                    for (int z = 0; z < 4; ++z) f1[p][0][z] = fo[p][k][z];
                }
                gemm<1, 2, NT, NT, true>(sq, f1, sadr + 2 * k * SG * kTile, Sh::kSl, SG, 2 * hf);
                gemm<1, 2, NT, NT, true>(sk, f2, sadr + 2 * k * SG * kTile, Sh::kSl, SG, 2 * hf);
                gemm<1, 2, NT, NT, true>(sc, f3, dadr + 2 * k * SG * kTile, Sh::kSl, SG, 2 * hf);
            }
            // <S_0, dS_1>: two elements of one row per turn
            for (int x = threadIdx.x; x < blocks * 16 * kSliceCols / 2; x += kGradThreads) {
                float2 s = make_float2(0, 0), d = make_float2(0, 0);
#pragma unroll
                for (int p = 0; p < NT; ++p) {
                    const uint8_t* base = ring + st * 2 * NT * Sh::kSl + p * Sh::kSl + x * 4;
                    const float2 s1 = unpack_h(*reinterpret_cast<const uint32_t*>(base));
                    const float2 d1 = unpack_h(*reinterpret_cast<const uint32_t*>(base + NT * Sh::kSl));
                    s.x += s1.x;
                    s.y += s1.y;
                    d.x += d1.x;
                    d.y += d1.y;
                }
                ss += (s.x * su) * (d.x * du) + (s.y * su) * (d.y * du);
            }
            // products with the chunk's own keys and queries
            float a1[2][4], a2[2][4], a3[2][4];
            zero(a1);
            zero(a2);
            zero(a3);
            const int t0 = n * SG + 2 * hf;       // column tile of the keys
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (k <= rb) {
                    uint32_t f1[NT][1][4], f2[NT][1][4];
#pragma unroll
                    for (int p = 0; p < NT; ++p) {
                        const uint32_t at = p * kSquare + ((2 * rb + (m8 & 1)) * 8 + 2 * k + (m8 >> 1)) * kTile + r8 * 16;
                        ldsm4(f1[p][0], pdadr + at);
                        ldsm4(f2[p][0], madr + at);
                    }
                    gemm<1, 2, NT, NT, true>(a1, f1, kadr + 2 * k * CG * kTile, Sh::kKey, CG, t0);
                    gemm<1, 2, NT, NT, true>(a2, f2, kadr + 2 * k * CG * kTile, Sh::kKey, CG, t0);
                }
                if (k >= rb) {
                    uint32_t f1[NT][1][4], f2[NT][1][4];
#pragma unroll
                    for (int p = 0; p < NT; ++p) {
                        const uint32_t at = p * kSquare + ((2 * k + (m8 >> 1)) * 8 + 2 * rb + (m8 & 1)) * kTile + r8 * 16;
                        ldsm4t(f1[p][0], pdadr + at);
                        ldsm4t(f2[p][0], madr + at);
                    }
                    gemm<1, 2, NT, NT, true>(a3, f1, qadr + 2 * k * CG * kTile, Sh::kKey, CG, t0);
                    gemm<1, 2, NT, NT, true>(a2, f2, kadr + 2 * k * CG * kTile, Sh::kKey, CG, t0);
                }
            }
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int i = i0 + 8 * h;
                    float2 kx = make_float2(0, 0), qx = make_float2(0, 0);
#pragma unroll
                    for (int p = 0; p < NT; ++p) {
                        const int at = p * Sh::kKey + ((2 * rb + h) * CG + t0 + t) * kTile + lane * 4;
                        const float2 k1 = unpack_h(*reinterpret_cast<const uint32_t*>(kimg + at));
                        const float2 q1 = unpack_h(*reinterpret_cast<const uint32_t*>(qimg + at));
                        kx.x += k1.x;
                        kx.y += k1.y;
                        qx.x += q1.x;
                        qx.y += q1.y;
                    }
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const float kz = z ? kx.y : kx.x, qz = z ? qx.y : qx.x;
                        const float q = times_pow2(sq[t][2 * h + z], q_exp) * gam[i];
                        const float k = times_pow2(sk[t][2 * h + z], k_exp) * -gam[i];     // without beta
                        const float c = times_pow2(sc[t][2 * h + z], c_exp) * rest[i];
                        dotq[h] += qz * q;
                        dotk[h] += kz * k;
                        dotc[h] += kz * c;
                        dq[n][t][2 * h + z] += q + pd_inv * a1[t][2 * h + z];
                        dkk[n][t][2 * h + z] += beta[i] * k + c + m_inv * a2[t][2 * h + z] + pd_inv * a3[t][2 * h + z];
                    }
                }
            __syncthreads();       // the slice is done with
            if (threadIdx.x == 0 && n + Sh::kRing < SL) copy_slice(head, n + Sh::kRing);
        }
        // sums over the row's lanes, then over halves
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[6] = {rn[h], rbeta[h], dotq[h], dotk[h], dotc[h], rv[h]};
#pragma unroll
            for (int x = 0; x < 6; ++x) {
                v[x] += __shfl_xor_sync(0xffffffffu, v[x], 1);
                v[x] += __shfl_xor_sync(0xffffffffu, v[x], 2);
                if ((lane & 3) == 0) sums[(hf * 6 + x) * kChunk + i0 + 8 * h] = v[x];
            }
        }
        ss = warp_sum(ss);
        if (lane == 0) wsum[warp] = ss;
        if (!ok) s_at[2] = 1;
        __syncthreads();
        if (warp == 0) {
            float dG[2], dots = 0.0f;
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const int i = 2 * lane + z;
                auto row = [&](int x) { return sums[x * kChunk + i] + sums[(6 + x) * kChunk + i]; };
                const float q = row(R_Q), k = row(R_K);
                dots += q + beta[i] * k;
                dG[z] = row(R_N) - ((colsum[i] + colsum[kChunk + i]) + (colsum[2 * kChunk + i] + colsum[3 * kChunk + i])) +
                        (q + beta[i] * k) - row(R_COL);
                const float kap = pow2_inv(vec[V_KINV * kChunk + i]);
                if (i < rows && s_at[2] == 0)
                    static_cast<float*>(a.grads.dbeta)[(tok + i) * a.grads.beta_stride + head] =
                        (row(R_RV) + k + row(R_BETA)) * kap * kap;
            }
            float sdot = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sdot += wsum[i];
            const float total = gam[kChunk - 1] * sdot + warp_sum(dots);
            float run = dG[0] + dG[1];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float up = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += up;
            }
            float before = __shfl_up_sync(0xffffffffu, run, 1);
            if (lane == 0) before = 0.0f;
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const int i = 2 * lane + z;
                if (i < rows && s_at[2] == 0)
                    static_cast<float*>(a.grads.dg)[(tok + i) * a.grads.g_stride + head] =
                        total - (z ? before + dG[0] : before);
            }
        }
        if (g + 1 < group) {
            __syncthreads();
            if (threadIdx.x == 0) {
                copy_head(head + 1);
                for (int n = 0; n < Sh::kRing && n < SL; ++n) copy_slice(head + 1, n);
            }
        }
    }
    __syncthreads();
    if (s_at[2]) {
        if (threadIdx.x == 0) atomicAdd(a.status + OFRL_STAT_TIMEOUT, 1);
        return;
    }
#pragma unroll
    for (int n = 0; n < SL; ++n)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = rb * 16 + row4 + 8 * h, c = n * kSliceCols + (2 * hf + t) * 8 + col2;
                if (i >= rows || c >= dk) continue;
                const float qi = vec[V_QINV * kChunk + i], ki = vec[V_KINV * kChunk + i];
                float* pq = static_cast<float*>(a.grads.dq) + (tok + i) * a.grads.q_stride + (int64_t)khead * dk + c;
                float* pk = static_cast<float*>(a.grads.dk) + (tok + i) * a.grads.k_stride + (int64_t)khead * dk + c;
                pq[0] = dq[n][t][2 * h] * qi;
                pq[1] = dq[n][t][2 * h + 1] * qi;
                pk[0] = dkk[n][t][2 * h] * ki;
                pk[1] = dkk[n][t][2 * h + 1] * ki;
            }
}

template <int DK, int DV>
cudaError_t run(const GradArgs& g, int64_t grid, cudaStream_t st) {
    constexpr int smem = GradShared<DK, DV>::kBytes;
    static_assert(smem <= 227 * 1024, "shared memory");
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = opt_in(delta_grad_kernel<DK, DV>, smem, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(delta_grad_kernel<DK, DV>, dim3((unsigned)grid), dim3(kGradThreads), smem, st, g);
}

cudaError_t pick(const GradArgs& g, int64_t grid, cudaStream_t st) {
    if (g.shape.k_dim > 64) return g.shape.v_dim > 64 ? run<128, 128>(g, grid, st) : run<128, 64>(g, grid, st);
    return g.shape.v_dim > 64 ? run<64, 128>(g, grid, st) : run<64, 64>(g, grid, st);
}

}  // namespace

cudaError_t launch_grad(const SeqLaunch& a, const Prepared& p, const Images& fwd, const Images& rev, cudaStream_t st) {
    GradArgs g;
    g.shape = a.shape;
    g.in = a.in;
    g.ends = a.ends;
    g.episodes = a.episodes;
    g.keys = p.keys;
    g.pairs = p.pairs;
    g.s_img = fwd.state;
    g.u_img = fwd.vec;
    g.d_img = rev.state;
    g.r_img = rev.vec;
    g.s_unit = fwd.state_unit;
    g.u_unit = fwd.vec_unit;
    g.d_unit = rev.state_unit;
    g.r_unit = rev.vec_unit;
    g.dout = a.dout;
    g.grads = a.grads;
    g.status = a.status;
    const int64_t grid = slots_of(a.in.tokens, a.episodes) * a.shape.k_heads;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    return pick(g, grid, st);
}

}  // namespace delta
}  // namespace ofrl
