// Gradients of q, k, log decay and write strength for bf16 tokens, on tcgen05
// (delta_grad.cu has the formulas and does the same for fp32 tokens, whose
// two-plane operands do not fit beside each other in shared memory).
//
// One CTA of eight warps per (chunk, key head), looping over the group's
// value heads.  Accumulator rows are tokens twice: rows 0 .. 63 belong to dq,
// rows 64 .. 127 to dk, so each of these is one 128-row product:
//   N   = [dO; R] U^T                 (64 columns)
//   ST  = [dO; R] S_0                 (DK columns)
//   SC  = [ . ; U] dS_1
//   IN  = [PD; E] K,   PD_ij = D_ij N1_ij (j <= i),  E_ij = -D_ij N2_ij (j < i)
//   COL = [ . ; PD^T] Q + [ . ; M^T] K,   M_ij = beta_i E_ij
// ( . : rows whose results nobody reads; the operand's rows there are whatever
// shared memory holds).  Then, row by row,
//   dq = gamma ST_q + IN_q
//   dk = -gamma beta ST_k + beta IN_k + COL + rest SC
//   dbeta = R v + k (-gamma ST_k + IN_k)
//   dG = q dq + k (-gamma beta ST_k + beta IN_k) - k (COL + rest SC)
// with every dot product taken from the accumulators: the row sums and column
// sums of PD_ij q_i k_j then come from the same rounded PD and cancel.
// Thread = row and half of the columns.

#include "delta_mma.cuh"

namespace ofrl {
namespace delta {
namespace {

constexpr int kThreads = 256;
constexpr uint64_t kWaitNs = 1000000000ull;

struct GradTcArgs {
    ofrl_delta_shape shape;
    ofrl_delta_tokens in;
    const int32_t* ends;
    int32_t episodes;
    const uint8_t* keys;
    const uint8_t* pairs;
    const uint8_t *s_img, *u_img, *d_img, *r_img;
    const float *s_unit, *u_unit, *d_unit, *r_unit;
    const __nv_bfloat16* dout;
    ofrl_delta_grads grads;
    int32_t* status;
};

template <int DK, int DV>
struct Lay {
    static constexpr int kKey = kChunk * DK * 2;        // one of K^, Q^
    static constexpr int kVec = DV * kChunk * 2;        // one of U^T, R^T; half of an A image
    static constexpr int kState = DV * DK * 2;
    // [ . ; X] operands start 8 column groups before X: what lies there is
    // read, so X sits behind buffers at least that large
    static constexpr int off_au = 0;                    // [dO; R] for N
    static constexpr int off_as = off_au + 2 * kVec;    // [dO; R] for ST
    static constexpr int off_uh = off_as + 2 * kVec;    // U for SC
    static constexpr int off_u = off_uh + kVec;         // U^T as it came
    static constexpr int off_s = off_u + kVec;
    static constexpr int off_d = off_s + kState;
    static constexpr int off_k = off_d + kState;        // K^, Q^
    static constexpr int off_pem = off_k + 2 * kKey;    // PD, E, M: [8 column groups][24 row groups]
    static constexpr int kPem = 8 * 24 * kTile;
    static constexpr int off_vec = off_pem + kPem;
    static constexpr int off_sum = off_vec + kVecBytes;
    static constexpr int kBytes = off_sum + (2 * 4 * kChunk + 64) * 4;
    static_assert(off_pem >= 8 * 24 * kTile, "rows before PD");
    // TMEM columns
    static constexpr int t_st = 0, t_in = DK, t_sc = 2 * DK, t_n = 3 * DK;
    static constexpr int kCols = 3 * DK + kChunk <= 256 ? 256 : 512;
};

__device__ __forceinline__ int exponent(float pow2) { return (int)((__float_as_uint(pow2) >> 23) & 255u) - 127; }
__device__ __forceinline__ float pow2f(int e) {
    return __uint_as_float((uint32_t)(min(max(e, -126), 127) + 127) << 23);
}
__device__ __forceinline__ uint32_t half_pow2(int e) {      // two halves 2^e, e <= 0
    const uint32_t h = e >= -14 ? (uint32_t)(e + 15) << 10 : e >= -24 ? 1u << (e + 24) : 0u;
    return h | h << 16;
}
__device__ __forceinline__ uint32_t mul_h2(uint32_t x, uint32_t f) {
    const __half2 p = __hmul2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&f));
    return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ uint4 mul_h8(uint4 x, uint32_t f) {
    return make_uint4(mul_h2(x.x, f), mul_h2(x.y, f), mul_h2(x.z, f), mul_h2(x.w, f));
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
    umma::tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// Operands along K (16 per instruction): a, b advance by the given bytes.
__device__ __forceinline__ void mma_run(uint32_t d, uint32_t a, uint32_t a_lbo, uint32_t a_sbo, uint32_t a_step,
                                        uint32_t b, uint32_t b_lbo, uint32_t b_sbo, uint32_t b_step, uint32_t idesc,
                                        int steps, bool accumulate) {
    for (int k = 0; k < steps; ++k)
        umma::mma_f16(d, umma::smem_desc(a + k * a_step, a_lbo, a_sbo), umma::smem_desc(b + k * b_step, b_lbo, b_sbo),
                      idesc, (accumulate || k > 0) ? 1u : 0u);
}

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads, DK == 64 && DV == 64 ? 2 : 1)
delta_grad_tc_kernel(const __grid_constant__ GradTcArgs a) {
    using L = Lay<DK, DV>;
    constexpr int CG = DK / 8, VB = DV / 16, VM = DV / 64, H = DK / 2;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bar_keys, bar_head, bar_n, bar_s, bar_i, bar_c;
    __shared__ uint32_t s_tmem;
    __shared__ int s_at[3];
    __shared__ float s_unit[4][8];          // powers of two of S_0, U, dS_1, R
    __shared__ int s_oexp[8];               // of dO per 8 tokens
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hk = a.shape.k_heads, hv = a.shape.v_heads, group = hv / hk, dk = a.shape.k_dim, dv = a.shape.v_dim;
    const int64_t slot = blockIdx.x / hk;
    const int khead = blockIdx.x % hk;
    if (warp == 0) {
        const int32_t tokens = (int32_t)a.in.tokens;
        const int e = episode_of(a.ends, a.episodes, tokens, (int32_t)slot);
        const Span sp = span_of(a.ends, e, tokens);
        const int c = (int)slot - (sp.start / kChunk + e);
        if (lane == 0) {
            s_at[0] = sp.start + c * kChunk;
            s_at[1] = c < 0 ? 0 : min(sp.len - c * kChunk, kChunk);
            s_at[2] = 0;
            umma::mbar_init(&bar_keys, 1);
            umma::mbar_init(&bar_head, 1);
            umma::mbar_init(&bar_n, 1);
            umma::mbar_init(&bar_s, 1);
            umma::mbar_init(&bar_i, 1);
            umma::mbar_init(&bar_c, 1);
            umma::fence_mbar_init();
        }
    }
    __syncthreads();
    const int rows = s_at[1];
    if (rows <= 0) return;
    const int64_t tok = s_at[0], at0 = slot * hv;
    const int blocks = (dv + 15) / 16;
    uint8_t *au = smem + L::off_au, *as = smem + L::off_as, *uh = smem + L::off_uh, *pem = smem + L::off_pem;
    const uint8_t *kimg = smem + L::off_k, *qimg = kimg + L::kKey;
    const uint32_t base = umma::smem_u32(smem);
    float* vec = reinterpret_cast<float*>(smem + L::off_vec);
    float* sums = reinterpret_cast<float*>(smem + L::off_sum);      // [2 halves][4][64]
    float* red = sums + 2 * 4 * kChunk;                             // [64]
    enum { R_Q, R_ST, R_IN, R_COL };

    auto copy_head = [&](int head) {
        umma::mbar_expect_tx(&bar_head, L::kVec + 2 * L::kState + kVecBytes);
        umma::bulk_g2s(vec, a.pairs + (at0 + head) * kPairBytes + 2 * kSquare, kVecBytes, &bar_head);
        umma::bulk_g2s(smem + L::off_u, a.u_img + (at0 + head) * L::kVec, L::kVec, &bar_head);
        umma::bulk_g2s(smem + L::off_s, a.s_img + (at0 + head) * L::kState, L::kState, &bar_head);
        umma::bulk_g2s(smem + L::off_d, a.d_img + (at0 + head) * L::kState, L::kState, &bar_head);
    };
    if (threadIdx.x == 0) {
        umma::mbar_expect_tx(&bar_keys, 2 * L::kKey);
        umma::bulk_g2s(smem + L::off_k, a.keys + (slot * hk + khead) * KeyImage::bytes(DK, 1), 2 * L::kKey, &bar_keys);
        copy_head(khead * group);
    }
    if (warp == 1) umma::tmem_alloc(&s_tmem, L::kCols);
    bool ok = true;

    auto wait_mma = [&](uint64_t* bar, int turn) {
        ok &= umma::mbar_wait(bar, (uint32_t)turn & 1u, kWaitNs);
        __syncwarp();
        umma::fence_after_sync();
    };
    const int row = (warp & 3) * 32 + lane;      // accumulator row
    const int i = row & 63, half = warp >> 2;    // token, column half
    const bool isk = row >= 64;
    float acc[H];
#pragma unroll
    for (int c = 0; c < H; ++c) acc[c] = 0.0f;

    for (int g = 0; g < group; ++g) {
        const int head = khead * group + g;
        // what this warp converts: tokens 8 warp .. + 7, channels 2 lane, + 1 of every 64
        uint32_t xo[VM][8], xv[VM][8];
        uint4 xr[VM][2];
        {
            const __nv_bfloat16* po = a.dout + (tok * hv + head) * dv;
            const __nv_bfloat16* pv = static_cast<const __nv_bfloat16*>(a.in.v) + tok * a.in.v_stride + (int64_t)head * dv;
            const uint8_t* pr = a.r_img + (at0 + head) * L::kVec;
#pragma unroll
            for (int m = 0; m < VM; ++m) {
                const int ch = m * 64 + 2 * lane;
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    const int j = warp * 8 + t;
                    const bool on = j < rows && ch < dv;
                    xo[m][t] = on ? *reinterpret_cast<const uint32_t*>(po + (int64_t)j * hv * dv + ch) : 0u;
                    xv[m][t] = on ? *reinterpret_cast<const uint32_t*>(pv + j * a.in.v_stride + ch) : 0u;
                }
#pragma unroll
                for (int z = 0; z < 2; ++z)
                    xr[m][z] = ch < blocks * 16
                                   ? *reinterpret_cast<const uint4*>(pr + ((ch >> 3) * 8 + warp) * kTile + ((ch + z) & 7) * 16)
                                   : make_uint4(0, 0, 0, 0);
            }
        }
        if (threadIdx.x < 32) {
            const float* p = threadIdx.x < 8    ? a.s_unit
                             : threadIdx.x < 16 ? a.u_unit
                             : threadIdx.x < 24 ? a.d_unit
                                                : a.r_unit;
            const int b = threadIdx.x & 7;
            s_unit[threadIdx.x >> 3][b] = b < blocks ? p[(at0 + head) * 8 + b] : 0.0f;
        }
        ok &= umma::mbar_wait(&bar_head, (uint32_t)g & 1u, kWaitNs);
        __syncthreads();
        const float *gam = vec + V_GAM * kChunk, *rest = vec + V_REST * kChunk, *beta = vec + V_BETA * kChunk;
        const float *ghi = vec + V_GHI * kChunk, *glo = vec + V_GLO * kChunk;
        // exponents of the products' units: the largest, and below it per block
        int top_o = -1000, top_os = -1000, top_r = -1000, top_rs = -1000, top_c = -1000;
#pragma unroll
        for (int b = 0; b < VB; ++b)
            if (b < blocks) {
                const int es = exponent(s_unit[0][b]), eu = exponent(s_unit[1][b]), ed = exponent(s_unit[2][b]),
                          er = exponent(s_unit[3][b]);
                top_o = max(top_o, eu);
                top_os = max(top_os, es);
                top_r = max(top_r, eu + er);
                top_rs = max(top_rs, es + er);
                top_c = max(top_c, ed + eu);
            }
        {
            float mx = 0.0f, qs[8];
#pragma unroll
            for (int t = 0; t < 8; ++t) qs[t] = vec[V_QS * kChunk + warp * 8 + t];
#pragma unroll
            for (int m = 0; m < VM; ++m)
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    const float2 x = unpack_b(xo[m][t]);
                    mx = fmaxf(mx, fmaxf(fabsf(x.x * qs[t]), fabsf(x.y * qs[t])));
                }
            const float up = scale_up(warp_max(mx));
            if (lane == 0) s_oexp[warp] = -exponent(up);
            float rv[8];
#pragma unroll
            for (int t = 0; t < 8; ++t) rv[t] = 0.0f;
#pragma unroll
            for (int m = 0; m < VM; ++m) {
                const int ch = m * 64 + 2 * lane, b = ch >> 4;
                if (ch >= blocks * 16) continue;
                const int es = exponent(s_unit[0][b]), eu = exponent(s_unit[1][b]), ed = exponent(s_unit[2][b]),
                          er = exponent(s_unit[3][b]);
                const uint32_t fo = half_pow2(eu - top_o), fos = half_pow2(es - top_os), fr = half_pow2(eu + er - top_r),
                               frs = half_pow2(es + er - top_rs), fc = half_pow2(ed + eu - top_c);
                const float ru = s_unit[3][b];
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    uint32_t h[4];
#pragma unroll
                    for (int t = 0; t < 8; t += 2) {
                        const float2 x0 = unpack_b(xo[m][t]), x1 = unpack_b(xo[m][t + 1]);
                        h[t / 2] = pack_h((z ? x0.y : x0.x) * (qs[t] * up), (z ? x1.y : x1.x) * (qs[t + 1] * up));
                    }
                    const uint4 o = make_uint4(h[0], h[1], h[2], h[3]);
                    const int rg = ch >> 3, r = (ch + z) & 7;
                    const int at_o = (warp * (DV / 8) + rg) * kTile + r * 16, at_r = ((8 + warp) * (DV / 8) + rg) * kTile + r * 16;
                    *reinterpret_cast<uint4*>(au + at_o) = mul_h8(o, fo);
                    *reinterpret_cast<uint4*>(as + at_o) = mul_h8(o, fos);
                    *reinterpret_cast<uint4*>(au + at_r) = mul_h8(xr[m][z], fr);
                    *reinterpret_cast<uint4*>(as + at_r) = mul_h8(xr[m][z], frs);
                    const uint4 u = *reinterpret_cast<const uint4*>(smem + L::off_u + (rg * 8 + warp) * kTile + r * 16);
                    *reinterpret_cast<uint4*>(uh + at_o) = mul_h8(u, fc);
                    const uint32_t w[4] = {xr[m][z].x, xr[m][z].y, xr[m][z].z, xr[m][z].w};
#pragma unroll
                    for (int t = 0; t < 8; ++t) {
                        const float2 rr = unpack_h(w[t / 2]), v = unpack_b(xv[m][t]);
                        rv[t] += (t & 1 ? rr.y : rr.x) * ru * (z ? v.y : v.x);
                    }
                }
            }
            // sums over the warp's lanes: lane l ends with token l & 7's
#pragma unroll
            for (int o = 4, n = 4; n >= 1; o >>= 1, n >>= 1) {
                const bool up2 = (lane & o) != 0;
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    if (t < n) {
                        const float keep = up2 ? rv[t + n] : rv[t], give = up2 ? rv[t] : rv[t + n];
                        rv[t] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                    }
            }
            rv[0] += __shfl_xor_sync(0xffffffffu, rv[0], 8);
            rv[0] += __shfl_xor_sync(0xffffffffu, rv[0], 16);
            if (lane < 8) red[warp * 8 + lane] = rv[0];      // R v, v unscaled
        }
        umma::fence_smem_to_async();
        umma::fence_before_sync();
        __syncthreads();
        umma::fence_after_sync();
        const uint32_t tmem = s_tmem;
        if (threadIdx.x == 0) {
            if (g == 0) ok &= umma::mbar_wait(&bar_keys, 0, kWaitNs);
            const uint32_t id_n = umma::instr_desc(umma::kTypeF16, true, true, 128, kChunk);
            const uint32_t id_s = umma::instr_desc(umma::kTypeF16, true, true, 128, DK);
            constexpr uint32_t kA = (DV / 8) * kTile;       // A images: column groups of tokens
            mma_run(tmem + L::t_n, base + L::off_au, kTile, kA, 2 * kTile, base + L::off_u, 8 * kTile, kTile,
                    2 * 8 * kTile, id_n, blocks, false);
            umma::commit(&bar_n);
            mma_run(tmem + L::t_st, base + L::off_as, kTile, kA, 2 * kTile, base + L::off_s, CG * kTile, kTile,
                    2 * CG * kTile, id_s, blocks, false);
            mma_run(tmem + L::t_sc, base + L::off_uh - 8 * kA, kTile, kA, 2 * kTile, base + L::off_d, CG * kTile, kTile,
                    2 * CG * kTile, id_s, blocks, false);
            umma::commit(&bar_s);
        }
        // <S_0, dS_1> meanwhile: 8 elements of one row per turn
        float ss = 0.0f;
        for (int x = threadIdx.x; x < blocks * 2 * CG * 8; x += kThreads) {
            const int b = x / (2 * CG * 8);
            const uint4 s = reinterpret_cast<const uint4*>(smem + L::off_s)[x], d = reinterpret_cast<const uint4*>(smem + L::off_d)[x];
            const uint32_t sw[4] = {s.x, s.y, s.z, s.w}, dw[4] = {d.x, d.y, d.z, d.w};
            float p = 0.0f;
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const float2 f = unpack_h(sw[z]), h = unpack_h(dw[z]);
                p += f.x * h.x + f.y * h.y;
            }
            ss += p * s_unit[0][b] * s_unit[2][b];
        }
        ss = warp_sum(ss);

        // N -> PD, E, M
        wait_mma(&bar_n, g);
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        float n[32];
        tmem_ld32(lanes + L::t_n + half * 32, n);
        const int oexp = s_oexp[i >> 3];
        {
            const int e = isk ? top_r : top_o + oexp;
            const float f1 = pow2f(e / 2), f2 = (isk ? -1.0f : 1.0f) * pow2f(e - e / 2);
            const float gi = ghi[i], li = glo[i];
#pragma unroll
            for (int c = 0; c < 32; ++c) {
                const int j = half * 32 + c;
                const bool in = isk ? j < i : j <= i;
                n[c] = in ? n[c] * f1 * f2 * exp2f((gi - ghi[j]) + (li - glo[j])) : 0.0f;
            }
        }
        const float bi = beta[i];
        float mx = 0.0f;
#pragma unroll
        for (int c = 0; c < 32; ++c) mx = fmaxf(mx, fabsf(n[c]));
        {
            // warps of dk rows: E for IN, M = beta E for COL together with PD
            const float m1 = warp_max(isk ? fabsf(bi) * mx : mx), m2 = warp_max(mx);
            if (lane == 0) {
                sums[warp * 3] = m1;
                sums[warp * 3 + 1] = isk ? m2 : 0.0f;
                sums[warp * 3 + 2] = ss;
            }
        }
        __syncthreads();
        float m1 = 0.0f, m2 = 0.0f, sdot = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            m1 = fmaxf(m1, sums[w * 3]);
            m2 = fmaxf(m2, sums[w * 3 + 1]);
            sdot += sums[w * 3 + 2];
        }
        const float p_up = scale_up(m1), p_inv = pow2_inv(p_up), e_up = scale_up(m2), e_inv = pow2_inv(e_up);
        {
            const int rg = row >> 3, r = row & 7;
            const float s1 = isk ? e_up : p_up, s2 = bi * p_up;
#pragma unroll
            for (int c = 0; c < 32; c += 8) {
                const int cg = half * 4 + c / 8;
                uint4 v = make_uint4(pack_h(n[c] * s1, n[c + 1] * s1), pack_h(n[c + 2] * s1, n[c + 3] * s1),
                                     pack_h(n[c + 4] * s1, n[c + 5] * s1), pack_h(n[c + 6] * s1, n[c + 7] * s1));
                *reinterpret_cast<uint4*>(pem + (cg * 24 + rg) * kTile + r * 16) = v;
                if (isk) {
                    v = make_uint4(pack_h(n[c] * s2, n[c + 1] * s2), pack_h(n[c + 2] * s2, n[c + 3] * s2),
                                   pack_h(n[c + 4] * s2, n[c + 5] * s2), pack_h(n[c + 6] * s2, n[c + 7] * s2));
                    *reinterpret_cast<uint4*>(pem + (cg * 24 + 8 + rg) * kTile + r * 16) = v;
                }
            }
        }
        umma::fence_smem_to_async();
        umma::fence_before_sync();
        __syncthreads();
        umma::fence_after_sync();
        constexpr uint32_t kP = 24 * kTile;
        if (threadIdx.x == 0) {
            const uint32_t id = umma::instr_desc(umma::kTypeF16, false, true, 128, DK);
            mma_run(tmem + L::t_in, base + L::off_pem, kP, kTile, 2 * kP, base + L::off_k, CG * kTile, kTile,
                    2 * CG * kTile, id, 4, false);
            umma::commit(&bar_i);
        }

        // this thread's row of q^ (dq rows) or k^ (dk rows), its half of the channels
        const uint8_t* xrow = (isk ? kimg : qimg) + ((i >> 3) * CG + half * (CG / 2)) * kTile + (i & 7) * 16;
        auto dot_row = [&](const float (&v)[32], int c0) {
            float d = 0.0f;
#pragma unroll
            for (int c = 0; c < 32; c += 8) {
                const uint4 x = *reinterpret_cast<const uint4*>(xrow + (c0 + c) / 8 * kTile);
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const float2 f = unpack_h(w[z]);
                    d += f.x * v[c + 2 * z] + f.y * v[c + 2 * z + 1];
                }
            }
            return d;
        };
        const float gi = gam[i];
        float dst = 0.0f, din = 0.0f, dcol = 0.0f;
        wait_mma(&bar_s, g);
        {
            const int e = isk ? top_rs : top_os + oexp;
            const float f1 = pow2f(e / 2), f2 = (isk ? -gi : gi) * pow2f(e - e / 2), bm = isk ? bi : 1.0f;
            const int ec = top_c;
            const float c1 = pow2f(ec / 2), c2 = rest[i] * pow2f(ec - ec / 2);
#pragma unroll
            for (int c0 = 0; c0 < H; c0 += 32) {
                float v[32];
                tmem_ld32(lanes + L::t_st + half * H + c0, v);
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    v[c] = v[c] * f1 * f2;
                    acc[c0 + c] += bm * v[c];
                }
                dst += dot_row(v, c0);
                if (isk) {
                    tmem_ld32(lanes + L::t_sc + half * H + c0, v);
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        v[c] = v[c] * c1 * c2;
                        acc[c0 + c] += v[c];
                    }
                    dcol += dot_row(v, c0);
                }
            }
        }
        umma::fence_before_sync();
        __syncthreads();
        umma::fence_after_sync();
        if (threadIdx.x == 0) {
            const uint32_t id = umma::instr_desc(umma::kTypeF16, true, true, 128, DK);
            mma_run(tmem + L::t_st, base + L::off_pem - 8 * kP, kTile, kP, 2 * kTile, base + L::off_k + L::kKey,
                    CG * kTile, kTile, 2 * CG * kTile, id, 4, false);
            mma_run(tmem + L::t_st, base + L::off_pem + 16 * kTile - 8 * kP, kTile, kP, 2 * kTile, base + L::off_k,
                    CG * kTile, kTile, 2 * CG * kTile, id, 4, true);
            umma::commit(&bar_c);
        }
        wait_mma(&bar_i, g);
        {
            const float f = isk ? e_inv : p_inv, bm = isk ? bi : 1.0f;
#pragma unroll
            for (int c0 = 0; c0 < H; c0 += 32) {
                float v[32];
                tmem_ld32(lanes + L::t_in + half * H + c0, v);
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    v[c] *= f;
                    acc[c0 + c] += bm * v[c];
                }
                din += dot_row(v, c0);
            }
        }
        wait_mma(&bar_c, g);
        if (isk) {
#pragma unroll
            for (int c0 = 0; c0 < H; c0 += 32) {
                float v[32];
                tmem_ld32(lanes + L::t_st + half * H + c0, v);
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    v[c] *= p_inv;
                    acc[c0 + c] += v[c];
                }
                dcol += dot_row(v, c0);
            }
        }
        // [half][..][token]: q (dq), k (state part without beta), k (IN without beta), k (column part);
        // dq rows keep the state part apart as well
        if (!isk) {
            sums[(half * 4 + R_Q) * kChunk + i] = dst + din;
        } else {
            sums[(half * 4 + R_ST) * kChunk + i] = dst;
            sums[(half * 4 + R_IN) * kChunk + i] = din;
            sums[(half * 4 + R_COL) * kChunk + i] = dcol;
        }
        // sum over tokens of the state parts' dots, times beta for k
        const float sd = warp_sum(isk ? bi * dst : dst);
        __shared__ float s_part[8];
        if (lane == 0) s_part[warp] = sd;
        if (!ok) s_at[2] = 1;
        umma::fence_before_sync();
        __syncthreads();
        umma::fence_after_sync();
        if (warp == 0 && s_at[2] == 0) {
            float total = gam[kChunk - 1] * sdot;
#pragma unroll
            for (int w = 0; w < 8; ++w) total += s_part[w];
            float dG[2];
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const int t = 2 * lane + z;
                auto two = [&](int x) { return sums[x * kChunk + t] + sums[(4 + x) * kChunk + t]; };
                const float k0 = two(R_ST) + two(R_IN), kinv = vec[V_KINV * kChunk + t], kap = pow2_inv(kinv);
                dG[z] = two(R_Q) + beta[t] * k0 - two(R_COL);
                if (t < rows)
                    static_cast<__nv_bfloat16*>(a.grads.dbeta)[(tok + t) * a.grads.beta_stride + head] =
                        __float2bfloat16_rn((red[t] * kinv + k0) * kap * kap);
            }
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
                const int t = 2 * lane + z;
                if (t < rows)
                    static_cast<__nv_bfloat16*>(a.grads.dg)[(tok + t) * a.grads.g_stride + head] =
                        __float2bfloat16_rn(total - (z ? before + dG[0] : before));
            }
        }
        if (g + 1 < group) {
            __syncthreads();
            if (threadIdx.x == 0) copy_head(head + 1);
        }
    }
    if (s_at[2] == 0 && i < rows) {
        const float f = vec[(isk ? V_KINV : V_QINV) * kChunk + i];
        __nv_bfloat16* to = isk ? static_cast<__nv_bfloat16*>(a.grads.dk) + (tok + i) * a.grads.k_stride
                                : static_cast<__nv_bfloat16*>(a.grads.dq) + (tok + i) * a.grads.q_stride;
        to += (int64_t)khead * dk + half * H;
#pragma unroll
        for (int c = 0; c < H; c += 8)
            if (half * H + c < dk)
                *reinterpret_cast<uint4*>(to + c) =
                    make_uint4(pack_b(acc[c] * f, acc[c + 1] * f), pack_b(acc[c + 2] * f, acc[c + 3] * f),
                               pack_b(acc[c + 4] * f, acc[c + 5] * f), pack_b(acc[c + 6] * f, acc[c + 7] * f));
    }
    __syncthreads();
    if (s_at[2] && threadIdx.x == 0) atomicAdd(a.status + OFRL_STAT_TIMEOUT, 1);
    if (warp == 1) umma::tmem_dealloc(s_tmem, L::kCols);
}

template <int DK, int DV>
cudaError_t run(const GradTcArgs& g, int64_t grid, cudaStream_t st) {
    constexpr int smem = Lay<DK, DV>::kBytes;
    static_assert(smem <= 226 * 1024, "shared memory");
    cudaError_t e = cudaFuncSetAttribute(delta_grad_tc_kernel<DK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = set_max_shared_carveout(delta_grad_tc_kernel<DK, DV>);
    if (e != cudaSuccess) return e;
    delta_grad_tc_kernel<DK, DV><<<(unsigned)grid, kThreads, smem, st>>>(g);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_grad_tc(const SeqLaunch& a, const Prepared& p, const Images& fwd, const Images& rev, cudaStream_t st) {
    GradTcArgs g;
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
    g.dout = static_cast<const __nv_bfloat16*>(a.dout);
    g.grads = a.grads;
    g.status = a.status;
    const int64_t grid = slots_of(a.in.tokens, a.episodes) * a.shape.k_heads;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    if (a.shape.k_dim > 64) return a.shape.v_dim > 64 ? run<128, 128>(g, grid, st) : run<128, 64>(g, grid, st);
    return a.shape.v_dim > 64 ? run<64, 128>(g, grid, st) : run<64, 64>(g, grid, st);
}

}  // namespace delta
}  // namespace ofrl
