// Gradients of q, k, log decay and write strength for bf16 tokens, on tcgen05
// (delta_grad.cu has the formulas and does the same for fp32 tokens, whose
// two-plane operands do not fit beside each other in shared memory).
//
// Persistent CTAs of eight warps take (chunk, key head) items from a counter
// and loop over the group's value heads; the next head's operands are copied in
// while this one's results leave TMEM.  Accumulator rows are tokens twice: rows
// 0 .. 63 belong to dq, rows 64 .. 127 to dk, so each of these is one 128-row
// product:
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
//
// Bound by the latency from an item's copies to its results, little of which
// fits beside another item's in 227 KB of shared memory: 640 items of 64 x 64
// (16384 tokens) 23 us; 2504 pairs of 128-wide heads (65k ragged tokens) 204 us,
// 3.4 TB/s.  Sixteen warps a CTA spill (318 us); asking L2 for the next item's
// operands ahead of their copies took 9 us off.

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
    int64_t items;
    unsigned* next;      // zero at the start of the launch
    int num_sms;
    int32_t* status;
};

template <int DK, int DV>
struct Lay {
    static constexpr int kKey = kChunk * DK * 2;        // one of K^, Q^
    static constexpr int kVec = DV * kChunk * 2;        // U^T, or R^T, or dO^T
    static constexpr int kState = DV * DK * 2;
    // [ . ; X] operands start 8 column groups before X: what lies there is
    // read, so X sits behind buffers at least that large
    static constexpr int off_a = 0;                     // [dO; R]: column groups of tokens, row groups of channels
    static constexpr int off_u = off_a + 2 * kVec;      // U^T, likewise
    static constexpr int off_s = off_u + kVec;
    static constexpr int off_d = off_s + kState;
    static constexpr int off_k = off_d + kState;        // K^, Q^ of two items
    static constexpr int off_pem = off_k + 4 * kKey;    // PD, E, M: [8 column groups][24 row groups]
    static constexpr int kPem = 8 * 24 * kTile;          // (also where dq and dk are turned around)
    static_assert(kPem >= 8 * 32 * 80, "staging");
    static constexpr int off_vec = off_pem + kPem;      // of two heads
    static constexpr int off_sum = off_vec + 2 * kVecBytes;
    static constexpr int kBytes = off_sum + (2 * 4 * kChunk + 2 * kChunk) * 4;
    static_assert(off_pem >= 8 * 24 * kTile, "rows before PD");
    // TMEM columns
    static constexpr int t_st = 0, t_in = DK, t_sc = 2 * DK, t_n = 3 * DK;
    static constexpr int kCols = 3 * DK + kChunk <= 256 ? 256 : 512;
    static constexpr int kCtas = 2 * (kBytes + 2048) <= 227 * 1024 && kCols == 256 ? 2 : 1;
};

__device__ __forceinline__ int exponent(float pow2) { return (int)((__float_as_uint(pow2) >> 23) & 255u) - 127; }
__device__ __forceinline__ float pow2f(int e) {
    return __uint_as_float((uint32_t)(min(max(e, -126), 127) + 127) << 23);
}
// f 2^e, |e| <= 252.
__device__ __forceinline__ float times_pow2(float f, int e) { return f * pow2f(e / 2) * pow2f(e - e / 2); }
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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
    uint64_t da = umma::smem_desc(a, a_lbo, a_sbo), db = umma::smem_desc(b, b_lbo, b_sbo);
#pragma unroll 4
    for (int k = 0; k < steps; ++k) {      // the address field does not overflow: it holds 18 bits of bytes
        umma::mma_f16(d, da, db, idesc, (accumulate || k > 0) ? 1u : 0u);
        da += a_step >> 4;
        db += b_step >> 4;
    }
}

__device__ __forceinline__ void prefetch(const uint8_t* p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

struct Item {
    int64_t slot, tok;
    int khead, rows;      // rows 0: none left
};

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads, Lay<DK, DV>::kCtas) delta_grad_tc_kernel(const __grid_constant__ GradTcArgs a) {
    using L = Lay<DK, DV>;
    constexpr int CG = DK / 8, VM = DV / 64, H = DK / 2;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bar_keys, bar_head, bar_n, bar_s, bar_i, bar_c;
    __shared__ uint32_t s_tmem;
    __shared__ Item s_next;
    __shared__ int s_dead, s_oexp[8];       // exponents of dO per 8 tokens
    __shared__ float s_part[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hk = a.shape.k_heads, hv = a.shape.v_heads, group = hv / hk, dk = a.shape.k_dim, dv = a.shape.v_dim;
    const int blocks = (dv + 15) / 16;
    const uint32_t base = umma::smem_u32(smem);
    uint8_t *ado = smem + L::off_a, *pem = smem + L::off_pem;
    float* sums = reinterpret_cast<float*>(smem + L::off_sum);      // [2 halves][4][64]
    float* red = sums + 2 * 4 * kChunk;                             // [2][64] R v
    enum { R_Q, R_ST, R_IN, R_COL };

    // the next item with tokens, by one whole warp
    auto find = [&]() {
        Item it = {0, 0, 0, 0};
        while (true) {
            unsigned n = 0;
            if (lane == 0) n = atomicAdd(a.next, 1u);
            n = __shfl_sync(0xffffffffu, n, 0);
            if (n >= a.items) break;
            n = (unsigned)a.items - 1 - n;      // the backward chain's last images are still in L2
            it.slot = n / (unsigned)hk;
            it.khead = (int)(n % (unsigned)hk);
            const Chunk c = chunk_of(a.ends, a.episodes, (int32_t)a.in.tokens, (int32_t)it.slot);
            it.rows = c.rows;
            it.tok = c.tok;
            if (it.rows > 0) break;
            it.rows = 0;
        }
        if (lane == 0) s_next = it;
    };
    pdl_wait();      // what the backward chain leaves
    if (warp == 0) {
        find();
        if (lane == 0) {
            s_dead = 0;
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
    Item it = s_next;
    if (it.rows <= 0) return;
    if (warp == 1) umma::tmem_alloc(&s_tmem, L::kCols);

    auto copy_keys = [&](const Item& x, int turn) {
        umma::mbar_expect_tx(&bar_keys, 2 * L::kKey);
        umma::bulk_g2s(smem + L::off_k + (turn & 1) * 2 * L::kKey, a.keys + (x.slot * hk + x.khead) * KeyImage::bytes(DK, 1),
                       2 * L::kKey, &bar_keys);
    };
    auto copy_head = [&](const Item& x, int head, int turn) {
        const int64_t at = x.slot * hv + head;
        umma::mbar_expect_tx(&bar_head, 2 * L::kVec + 2 * L::kState + kVecBytes);
        umma::bulk_g2s(smem + L::off_vec + (turn & 1) * kVecBytes, a.pairs + at * kPairBytes + 2 * kSquare, kVecBytes, &bar_head);
        umma::bulk_g2s(smem + L::off_a + L::kVec, a.r_img + at * L::kVec, L::kVec, &bar_head);
        umma::bulk_g2s(smem + L::off_u, a.u_img + at * L::kVec, L::kVec, &bar_head);
        umma::bulk_g2s(smem + L::off_s, a.s_img + at * L::kState, L::kState, &bar_head);
        umma::bulk_g2s(smem + L::off_d, a.d_img + at * L::kState, L::kState, &bar_head);
    };
    // what this thread converts: tokens 8 warp .. + 7, channels 2 lane, + 1 of every 64
    uint32_t xo[VM][8], xv[VM][8];
    float un[4];      // powers of two of S_0, U, dS_1, R
    auto load_head = [&](const Item& x, int head) {
        const __nv_bfloat16* po = a.dout + (x.tok * hv + head) * dv;
        const __nv_bfloat16* pv = static_cast<const __nv_bfloat16*>(a.in.v) + x.tok * a.in.v_stride + (int64_t)head * dv;
#pragma unroll
        for (int m = 0; m < VM; ++m) {
            const int ch = m * 64 + 2 * lane;
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const int j = warp * 8 + t;
                const bool on = j < x.rows && ch < dv;
                xo[m][t] = on ? *reinterpret_cast<const uint32_t*>(po + (int64_t)j * hv * dv + ch) : 0u;
                xv[m][t] = on ? *reinterpret_cast<const uint32_t*>(pv + j * a.in.v_stride + ch) : 0u;
            }
        }
        const int64_t at = x.slot * hv + head;
        un[0] = a.s_unit[at];
        un[1] = a.u_unit[at];
        un[2] = a.d_unit[at];
        un[3] = a.r_unit[at];
    };
    auto ahead = [&](const Item& x, int head, bool keys) {      // by one whole warp
        const int64_t at = x.slot * hv + head;
        if (lane == 0) {
            if (keys) prefetch(a.keys + (x.slot * hk + x.khead) * KeyImage::bytes(DK, 1), 2 * L::kKey);
            prefetch(a.r_img + at * L::kVec, L::kVec);
            prefetch(a.u_img + at * L::kVec, L::kVec);
            prefetch(a.s_img + at * L::kState, L::kState);
            prefetch(a.d_img + at * L::kState, L::kState);
            prefetch(a.pairs + at * kPairBytes + 2 * kSquare, kVecBytes);
        }
        const __nv_bfloat16* po = a.dout + (x.tok * hv + head) * dv;
        const __nv_bfloat16* pv = static_cast<const __nv_bfloat16*>(a.in.v) + x.tok * a.in.v_stride + (int64_t)head * dv;
        for (int j = lane; j < x.rows; j += 32)
            for (int c = 0; c < dv; c += 64) {      // 128 bytes
                asm volatile("prefetch.global.L2 [%0];" ::"l"(po + (int64_t)j * hv * dv + c));
                asm volatile("prefetch.global.L2 [%0];" ::"l"(pv + j * a.in.v_stride + c));
            }
    };
    if (threadIdx.x == 0) {
        copy_keys(it, 0);
        copy_head(it, it.khead * group, 0);
    }
    load_head(it, it.khead * group);

    const int row = (warp & 3) * 32 + lane;      // accumulator row
    const int i = row & 63, half = warp >> 2;    // token, column half
    const bool isk = row >= 64;
    bool ok = true;
    auto wait = [&](uint64_t* bar, int turn) {
        ok &= umma::mbar_wait(bar, (uint32_t)turn & 1u, kWaitNs);
        __syncwarp();
        umma::fence_after_sync();
    };
    float acc[H];
    int turn = 0, g = 0;                         // heads taken; head of the group
    int items = 0;
    while (true) {
        const int head = it.khead * group + g;
        const bool last = g + 1 == group;
        if (g == 0) {
#pragma unroll
            for (int c = 0; c < H; ++c) acc[c] = 0.0f;
            wait(&bar_keys, items);
        }
        wait(&bar_head, turn);
        const float* vec = reinterpret_cast<const float*>(smem + L::off_vec + (turn & 1) * kVecBytes);
        const uint8_t *kimg = smem + L::off_k + (items & 1) * 2 * L::kKey, *qimg = kimg + L::kKey;
        const float *gam = vec + V_GAM * kChunk, *rest = vec + V_REST * kChunk, *beta = vec + V_BETA * kChunk;
        const float *ghi = vec + V_GHI * kChunk, *glo = vec + V_GLO * kChunk;
        const int es = exponent(un[0]), eu = exponent(un[1]), ed = exponent(un[2]), er = exponent(un[3]);
        const float s_d = un[0], d_d = un[2];
        {
            float mx = 0.0f, qs[8], rv[8];
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                qs[t] = vec[V_QS * kChunk + warp * 8 + t];
                rv[t] = 0.0f;
            }
#pragma unroll
            for (int m = 0; m < VM; ++m)
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    const float2 x = unpack_b(xo[m][t]);
                    mx = fmaxf(mx, fmaxf(fabsf(x.x), fabsf(x.y)) * fabsf(qs[t]));
                }
            const float up = scale_up(warp_max(mx));
            if (lane == 0) s_oexp[warp] = -exponent(up);
#pragma unroll
            for (int t = 0; t < 8; ++t) qs[t] *= up;
#pragma unroll
            for (int m = 0; m < VM; ++m) {
                const int ch = m * 64 + 2 * lane;
                if (ch >= blocks * 16) continue;
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    uint32_t h[4];
#pragma unroll
                    for (int t = 0; t < 8; t += 2) {
                        const float2 x0 = unpack_b(xo[m][t]), x1 = unpack_b(xo[m][t + 1]);
                        h[t / 2] = pack_h((z ? x0.y : x0.x) * qs[t], (z ? x1.y : x1.x) * qs[t + 1]);
                    }
                    uint8_t* to = ado + (warp * (DV / 8) + (ch >> 3)) * kTile + ((ch + z) & 7) * 16;
                    *reinterpret_cast<uint4*>(to) = make_uint4(h[0], h[1], h[2], h[3]);
                    const uint4 r = *reinterpret_cast<const uint4*>(to + L::kVec);
                    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                    for (int t = 0; t < 8; ++t) {
                        const float2 rr = unpack_h(w[t / 2]), v = unpack_b(xv[m][t]);
                        rv[t] += (t & 1 ? rr.y : rr.x) * (z ? v.y : v.x);
                    }
                }
            }
            // sums over the warp's lanes: lane l ends with token l & 7's
#pragma unroll
            for (int o = 4, n = 4; n >= 1; o >>= 1, n >>= 1) {
                const bool hi = (lane & o) != 0;
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    if (t < n) {
                        const float keep = hi ? rv[t + n] : rv[t], give = hi ? rv[t] : rv[t + n];
                        rv[t] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                    }
            }
            rv[0] += __shfl_xor_sync(0xffffffffu, rv[0], 8);
            rv[0] += __shfl_xor_sync(0xffffffffu, rv[0], 16);
            if (lane < 8) red[(turn & 1) * kChunk + warp * 8 + lane] = rv[0] * un[3];      // R v, v unscaled
        }
        umma::fence_smem_to_async();
        umma::fence_before_sync();
        __syncthreads();
        umma::fence_after_sync();
        const uint32_t tmem = s_tmem;
        constexpr uint32_t kA = (DV / 8) * kTile;       // bytes of a column group of tokens
        if (threadIdx.x == 0) {
            const uint32_t id_n = umma::instr_desc(umma::kTypeF16, true, true, 128, kChunk);
            const uint32_t id_s = umma::instr_desc(umma::kTypeF16, true, true, 128, DK);
            mma_run(tmem + L::t_n, base + L::off_a, kTile, kA, 2 * kTile, base + L::off_u, kTile, kA, 2 * kTile, id_n,
                    blocks, false);
            umma::commit(&bar_n);
            mma_run(tmem + L::t_st, base + L::off_a, kTile, kA, 2 * kTile, base + L::off_s, kTile, kA, 2 * kTile, id_s,
                    blocks, false);
            mma_run(tmem + L::t_sc, base + L::off_u - 8 * kA, kTile, kA, 2 * kTile, base + L::off_d, kTile, kA, 2 * kTile,
                    id_s, blocks, false);
            umma::commit(&bar_s);
        }
        if (warp == 1) {
            // where the next head's operands are, and into L2 with them: they
            // can be copied only when this head's products are through, and
            // HBM's latency under load is most of a head's time
            if (last) find();
            __syncwarp();
            const Item p = last ? s_next : it;
            if (p.rows > 0) ahead(p, p.khead * group + (last ? 0 : g + 1), last);
        }
        // <S_0, dS_1> meanwhile: 8 elements of one row per turn
        float ss = 0.0f;
        {
            constexpr int kAtOnce = 4;
            const uint4 *ps = reinterpret_cast<const uint4*>(smem + L::off_s), *pd = reinterpret_cast<const uint4*>(smem + L::off_d);
            float part[kAtOnce] = {};
            for (int x0 = threadIdx.x; x0 < DV * DK / 8; x0 += kAtOnce * kThreads) {
                uint4 sv[kAtOnce], dv4[kAtOnce];
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) {
                    const int x = x0 + k * kThreads;
                    const bool in = x < DV * DK / 8;
                    sv[k] = in ? ps[x] : make_uint4(0, 0, 0, 0);
                    dv4[k] = in ? pd[x] : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) {
                    const uint32_t sw[4] = {sv[k].x, sv[k].y, sv[k].z, sv[k].w}, dw[4] = {dv4[k].x, dv4[k].y, dv4[k].z, dv4[k].w};
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const float2 f = unpack_h(sw[z]), h = unpack_h(dw[z]);
                        part[k] += f.x * h.x + f.y * h.y;
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) ss += part[k];
        }
        ss = warp_sum(ss);

        // N -> PD, E, M
        wait(&bar_n, turn);
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        float n[32];
        tmem_ld32(lanes + L::t_n + half * 32, n);
        const int oexp = s_oexp[i >> 3];
        const float bi = beta[i];
        float mx = 0.0f;
        {
            const float f = times_pow2(isk ? -1.0f : 1.0f, eu + (isk ? er : oexp));
            const float gi = ghi[i], li = glo[i];
            const int most = (isk ? i : i + 1) - half * 32;     // columns of this half that count
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
                const float4 h4 = *reinterpret_cast<const float4*>(ghi + half * 32 + c);
                const float4 l4 = *reinterpret_cast<const float4*>(glo + half * 32 + c);
                const float gh[4] = {h4.x, h4.y, h4.z, h4.w}, gl[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    n[c + z] = c + z < most ? n[c + z] * f * ex2((gi - gh[z]) + (li - gl[z])) : 0.0f;
                    mx = fmaxf(mx, fabsf(n[c + z]));
                }
            }
        }
        {
            // warps of dk rows: E for IN, M = beta E for COL together with PD
            const float m1 = warp_max(isk ? fabsf(bi) * mx : mx), m2 = warp_max(mx);
            if (lane == 0) {
                sums[warp * 4] = m1;
                sums[warp * 4 + 1] = isk ? m2 : 0.0f;
                sums[warp * 4 + 2] = ss;
            }
        }
        __syncthreads();
        float m1 = 0.0f, m2 = 0.0f, sdot = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            const float4 x = reinterpret_cast<const float4*>(sums)[w];
            m1 = fmaxf(m1, x.x);
            m2 = fmaxf(m2, x.y);
            sdot += x.z;
        }
        sdot = sdot * s_d * d_d;
        const float p_up = scale_up(m1), p_inv = pow2_inv(p_up), e_up = scale_up(m2), e_inv = pow2_inv(e_up);
        constexpr uint32_t kP = 24 * kTile;
        {
            const float s1 = isk ? e_up : p_up, s2 = bi * p_up;
            uint8_t* to = pem + half * 4 * kP + (row >> 3) * kTile + (row & 7) * 16;
#pragma unroll
            for (int c = 0; c < 32; c += 8) {
                *reinterpret_cast<uint4*>(to + c / 8 * kP) =
                    make_uint4(pack_h(n[c] * s1, n[c + 1] * s1), pack_h(n[c + 2] * s1, n[c + 3] * s1),
                               pack_h(n[c + 4] * s1, n[c + 5] * s1), pack_h(n[c + 6] * s1, n[c + 7] * s1));
                if (isk)
                    *reinterpret_cast<uint4*>(to + c / 8 * kP + 8 * kTile) =
                        make_uint4(pack_h(n[c] * s2, n[c + 1] * s2), pack_h(n[c + 2] * s2, n[c + 3] * s2),
                                   pack_h(n[c + 4] * s2, n[c + 5] * s2), pack_h(n[c + 6] * s2, n[c + 7] * s2));
            }
        }
        umma::fence_smem_to_async();
        umma::fence_before_sync();
        __syncthreads();
        umma::fence_after_sync();
        const uint32_t kadr = umma::smem_u32(kimg);
        if (threadIdx.x == 0) {
            const uint32_t id = umma::instr_desc(umma::kTypeF16, false, true, 128, DK);
            mma_run(tmem + L::t_in, base + L::off_pem, kP, kTile, 2 * kP, kadr, CG * kTile, kTile, 2 * CG * kTile, id, 4,
                    false);
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
        const float gi = gam[i], bm = isk ? bi : 1.0f;
        float dst = 0.0f, din = 0.0f, dcol = 0.0f;
        wait(&bar_s, turn);
        {
            const float f = times_pow2(isk ? -gi : gi, es + (isk ? er : oexp)), fb = f * bm;
#pragma unroll
            for (int c0 = 0; c0 < H; c0 += 32) {
                float v[32];
                tmem_ld32(lanes + L::t_st + half * H + c0, v);
#pragma unroll
                for (int c = 0; c < 32; ++c) acc[c0 + c] += fb * v[c];
                dst += f * dot_row(v, c0);
            }
        }
        umma::fence_before_sync();
        __syncthreads();
        umma::fence_after_sync();
        // the products over channels are done: room for the next head's operands
        const Item nx = last ? s_next : it;
        const int nhead = nx.khead * group + (last ? 0 : g + 1);
        if (threadIdx.x == 0) {
            const uint32_t id = umma::instr_desc(umma::kTypeF16, true, true, 128, DK);
            mma_run(tmem + L::t_st, base + L::off_pem - 8 * kP, kTile, kP, 2 * kTile, kadr + L::kKey, CG * kTile, kTile,
                    2 * CG * kTile, id, 4, false);
            mma_run(tmem + L::t_st, base + L::off_pem + 16 * kTile - 8 * kP, kTile, kP, 2 * kTile, kadr, CG * kTile, kTile,
                    2 * CG * kTile, id, 4, true);
            umma::commit(&bar_c);
            if (nx.rows > 0) {
                copy_head(nx, nhead, turn + 1);
                if (last) copy_keys(nx, items + 1);
            }
        }
        if (nx.rows > 0) load_head(nx, nhead);
        wait(&bar_i, turn);
        {
            const float f = isk ? e_inv : p_inv, fb = f * bm;
#pragma unroll
            for (int c0 = 0; c0 < H; c0 += 32) {
                float v[32];
                tmem_ld32(lanes + L::t_in + half * H + c0, v);
#pragma unroll
                for (int c = 0; c < 32; ++c) acc[c0 + c] += fb * v[c];
                din += f * dot_row(v, c0);
            }
        }
        wait(&bar_c, turn);
        if (isk) {
            const float f = times_pow2(rest[i], ed + eu);
#pragma unroll
            for (int c0 = 0; c0 < H; c0 += 32) {
                float v[32], w[32];
                tmem_ld32(lanes + L::t_sc + half * H + c0, v);
                tmem_ld32(lanes + L::t_st + half * H + c0, w);
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    v[c] = v[c] * f + w[c] * p_inv;
                    acc[c0 + c] += v[c];
                }
                dcol += dot_row(v, c0);
            }
        }
        // [half][..][token]: q (dq), k (state part without beta), k (IN without beta), k (column part)
        if (!isk) {
            sums[(half * 4 + R_Q) * kChunk + i] = dst + din;
        } else {
            sums[(half * 4 + R_ST) * kChunk + i] = dst;
            sums[(half * 4 + R_IN) * kChunk + i] = din;
            sums[(half * 4 + R_COL) * kChunk + i] = dcol;
        }
        // sum over tokens of the state parts' dots, times beta for k
        const float sd = warp_sum(bm * dst);
        if (lane == 0) s_part[warp] = sd;
        if (!ok) s_dead = 1;
        umma::fence_before_sync();
        __syncthreads();
        umma::fence_after_sync();
        const bool dead = s_dead != 0;
        if (warp == 0 && !dead) {
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
                if (t < it.rows)
                    static_cast<__nv_bfloat16*>(a.grads.dbeta)[(it.tok + t) * a.grads.beta_stride + head] =
                        __float2bfloat16_rn((red[(turn & 1) * kChunk + t] * kinv + k0) * kap * kap);
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
                if (t < it.rows)
                    static_cast<__nv_bfloat16*>(a.grads.dg)[(it.tok + t) * a.grads.g_stride + head] =
                        __float2bfloat16_rn(total - (z ? before + dG[0] : before));
            }
        }
        if (last && !dead) {
            // 32 rows of 32 channels at a time, turned around in shared memory
            // (what IN and COL read is done with) for whole sectors
            const float f = vec[(isk ? V_KINV : V_QINV) * kChunk + i];
            uint8_t* stage = pem + warp * 32 * 80;
            const int64_t stride = isk ? a.grads.k_stride : a.grads.q_stride;
            const int row0 = (warp & 1) * 32;      // token of the warp's first row
            __nv_bfloat16* to = static_cast<__nv_bfloat16*>(isk ? a.grads.dk : a.grads.dq) + (it.tok + row0) * stride +
                                (int64_t)it.khead * dk + half * H;
#pragma unroll
            for (int c0 = 0; c0 < H; c0 += 32) {
#pragma unroll
                for (int c = 0; c < 32; c += 8)
                    *reinterpret_cast<uint4*>(stage + lane * 80 + c * 2) =
                        make_uint4(pack_b(acc[c0 + c] * f, acc[c0 + c + 1] * f), pack_b(acc[c0 + c + 2] * f, acc[c0 + c + 3] * f),
                                   pack_b(acc[c0 + c + 4] * f, acc[c0 + c + 5] * f), pack_b(acc[c0 + c + 6] * f, acc[c0 + c + 7] * f));
                __syncwarp();
                const int c = c0 + (lane & 3) * 8;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = k * 8 + (lane >> 2);
                    if (row0 + r < it.rows && half * H + c < dk)
                        *reinterpret_cast<uint4*>(to + r * stride + c) =
                            *reinterpret_cast<const uint4*>(stage + r * 80 + (lane & 3) * 16);
                }
                __syncwarp();
            }
        }
        ++turn;
        if (!last) {
            ++g;
        } else {
            it = nx;
            g = 0;
            ++items;
        }
        if (nx.rows <= 0) break;
        if (dead) {      // wind down: wait, within limits, for the copies in flight
            umma::mbar_wait(&bar_head, (uint32_t)turn & 1u, kWaitNs);
            if (last) umma::mbar_wait(&bar_keys, (uint32_t)items & 1u, kWaitNs);
            break;
        }
    }
    __syncthreads();
    if (s_dead && threadIdx.x == 0) atomicAdd(a.status + OFRL_STAT_TIMEOUT, 1);
    if (warp == 1) umma::tmem_dealloc(s_tmem, L::kCols);
}

template <int DK, int DV>
cudaError_t run(const GradTcArgs& g, cudaStream_t st) {
    constexpr int smem = Lay<DK, DV>::kBytes;
    static_assert(smem <= 226 * 1024, "shared memory");
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = opt_in(delta_grad_tc_kernel<DK, DV>, smem, done);
    if (e != cudaSuccess) return e;
    const int64_t most = (int64_t)g.num_sms * Lay<DK, DV>::kCtas;
    const unsigned grid = (unsigned)(g.items < most ? g.items : most);
    if (grid == 0) return cudaSuccess;
    return launch_pdl(delta_grad_tc_kernel<DK, DV>, dim3(grid), dim3(kThreads), smem, st, g);
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
    g.items = slots_of(a.in.tokens, a.episodes) * a.shape.k_heads;
    g.next = a.counter;
    g.num_sms = a.num_sms;
    if (a.shape.k_dim > 64) return a.shape.v_dim > 64 ? run<128, 128>(g, st) : run<128, 64>(g, st);
    return a.shape.v_dim > 64 ? run<64, 128>(g, st) : run<64, 64>(g, st);
}

}  // namespace delta
}  // namespace ofrl
