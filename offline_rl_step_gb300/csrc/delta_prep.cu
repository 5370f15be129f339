// Per chunk of 64 tokens, independently of every state: the power-of-two
// scaled keys and queries, the decays, P and T = (1 + A)^-1 (see
// delta_mma.cuh for what is left where).
//
// One CTA of four warps per (chunk, value head); the first of a group also
// leaves the group's keys and queries.  (One CTA per key head would load them
// once, but leaves a chunk's heads in a row: twice the latency, half the
// CTAs to hide it.)
//
// [Q; K] K^T is one 128 x 64 product on tcgen05, read back a row per thread:
// two warps make P's rows, two A's, while the decays are added up before.
//
// T.  1 + A is unit lower triangular with blocks of 16.  The diagonal blocks are
// inverted by forward substitution (a lane per column); then warp w makes T's
// block column w, transposed, block after block:
//   T_rw^T = -(sum_{s=w}^{r-1} T_sw^T A_rs^T) T_rr^T.
// T^T's blocks lie on and above the diagonal of the image that holds A's below
// it.  Substitution, not a series of powers of A: with correlated keys the
// powers grow before they cancel.  The block products use bf16 planes (two, or
// three where 22 bits are kept): T's elements have no bound known beforehand.
//
// Six CTAs share an SM's instruction cache at different places of a kernel
// that runs through once, so its loops stay rolled where the work is the same.
//
// Bound by the latency of that sequence: 16 thousand cycles a CTA, six at a
// time, the schedulers busy for half of them.  640 CTAs of 64-wide bf16 heads
// (16384 tokens) 15 us; 5008 of 128-wide ones (65k ragged tokens) 81 us, 3.0
// TB/s of HBM.  Keys and queries through registers before the decays: 101 us;
// decays in every warp and a diagonal block to each: 86.

#include "delta_mma.cuh"

namespace ofrl {
namespace delta {
namespace {

constexpr int kPrepThreads = 128;
constexpr uint64_t kWaitNs = 1000000000ull;

struct PrepArgs {
    ofrl_delta_shape shape;
    ofrl_delta_tokens in;
    const int32_t* ends;
    int32_t episodes;
    uint8_t* keys;
    uint8_t* pairs;
    int32_t* status;
};

// 16 bytes into shared memory behind the thread's back; zeros where !in.
__device__ __forceinline__ void cp16(uint32_t to, const void* from, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(in ? 16 : 0) : "memory");
}

// Eight elements as they lie in memory, 16 bytes in each place.
template <typename T>
struct Raw {
    uint4 v[sizeof(T) / 2];
    __device__ __forceinline__ void load(const uint8_t* p, int step) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = *reinterpret_cast<const uint4*>(p + i * step);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[sizeof(T) / 2 - 1].x, v[sizeof(T) / 2 - 1].y,
                               v[sizeof(T) / 2 - 1].z, v[sizeof(T) / 2 - 1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (sizeof(T) == 4) {
                x[i] = __uint_as_float(w[i]);
            } else {
                const float2 f = unpack_b(w[i / 2]);
                x[i] = i & 1 ? f.y : f.x;
            }
        }
    }
};

// Power of two, 2^-most to 2^most, that divides a row: its largest magnitude
// becomes [1, 2).  A key's is squared beside beta and stays within 2^60.
__device__ __forceinline__ float row_unit(float amax, int most) {
    const int e = (int)((__float_as_uint(amax) >> 23) & 255u);
    if (e == 255 || amax == 0.0f) return 1.0f;
    return __uint_as_float((uint32_t)min(max(e, 127 - most), 127 + most) << 23);
}

// Unevaluated pairs of floats for running sums of log decays: a difference
// of two such sums is then exact to fp32 whatever the sums' size.
struct Two {
    float h, l;
};
__device__ __forceinline__ Two two_add(Two a, Two b) {
    const float s = a.h + b.h, z = s - a.h;
    const float e = ((a.h - (s - z)) + (b.h - z)) + (a.l + b.l);
    const float h = s + e;
    return {h, e - (h - s)};
}
// g log2(e), log2(e) itself as a pair.
__device__ __forceinline__ Two two_log2(float g) {
    constexpr float kHi = 1.44269502e0f, kLo = 1.92596303e-8f;
    const float h = g * kHi;
    return {h, fmaf(g, kHi, -h) + g * kLo};
}

template <int NM>
__device__ __forceinline__ float exp_2(float x) {      // 2^-22 is enough for one plane
    if constexpr (NM == 2) return exp2f(x);
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename T, int DK, int NM>
struct PrepShared {
    static constexpr int NT = sizeof(T) == 4 ? 2 : 1, NB = NM + 1;      // NB: bf16 planes inside the inversion
    static constexpr int kKey = kChunk * DK * 2;
    // planes of Q^ and K^; afterwards, in the same place, A's blocks below the
    // diagonal with T^T's on and above it, and the diagonal blocks in fp32
    static constexpr int off_diag = NB * kSquare;
    static constexpr int kPitch = 20;      // floats between columns of a diagonal block
    static constexpr int kAfter = off_diag + 4 * 16 * kPitch * 4;
    static constexpr int off_vec = 2 * NT * kKey > kAfter ? 2 * NT * kKey : kAfter;
    static constexpr int kBytes = off_vec + kVecBytes + 2 * kChunk * 4;
};

// T: token type; DK: padded key width; NM: planes of T and P.
template <typename T, int DK, int NM>
__global__ void __launch_bounds__(kPrepThreads, NM == 1 ? 6 : 4) delta_prep_kernel(const __grid_constant__ PrepArgs a) {
    using Sh = PrepShared<T, DK, NM>;
    constexpr int NT = Sh::NT, NB = Sh::NB, CG = DK / 8, KS = DK / 16, kKey = Sh::kKey, kPitch = Sh::kPitch;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* aimg = smem;      // [plane][Q^, K^] before
    __shared__ __align__(8) uint64_t bar;
    __shared__ uint32_t s_tmem;
    float* diag = reinterpret_cast<float*>(smem + Sh::off_diag);
    float* vec = reinterpret_cast<float*>(smem + Sh::off_vec);
    float* kap = vec + V_COUNT * kChunk;
    float* kqv = kap + kChunk;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hk = a.shape.k_heads, hv = a.shape.v_heads, group = hv / hk, dk = a.shape.k_dim;
    const int64_t slot = blockIdx.x / hv;
    const int head = blockIdx.x % hv, khead = head / group;
    const int32_t tokens = (int32_t)a.in.tokens;
    // The chain that follows reads the caller's buffers before it waits for this
    // kernel: what came before has to be done when it is let go, below.
    pdl_wait();
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e < a.episodes; e += kPrepThreads)
            if (span_bad(a.ends, e, tokens)) atomicAdd(a.status + OFRL_STAT_BAD_INDEX, 1);
    const Chunk at = chunk_of(a.ends, a.episodes, tokens, (int32_t)slot);      // by every warp
    const int rows = at.rows;
    if (rows <= 0) return;
    const int64_t tok = at.tok;

    if (threadIdx.x == 0) {
        umma::mbar_init(&bar, 1);
        umma::fence_mbar_init();
    }
    if (warp == 3) {
        umma::tmem_alloc(&s_tmem, kChunk);
        // Only now may the chain start: on tcgen05 it takes all of an SM's TMEM
        // before it waits for this kernel, and a CTA here that had none yet would
        // wait for the chain in turn.  (So no other warp lets it go, either.)
        pdl_trigger();
    }
    // One warp adds up the decays and two invert the diagonal blocks; which ones
    // changes from CTA to CTA, so that every scheduler of an SM gets its share.
    const int chosen = (int)(blockIdx.x * 0x9E3779B1u >> 30);
    const bool adds = warp == chosen, inverts = (warp >> 1) == (chosen & 1);
    T gin[2], bin[2];      // tokens 2 lane, + 1 (past the end: the last one's, not used)
    if (adds)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t t = tok + min(2 * lane + i, rows - 1);
            gin[i] = static_cast<const T*>(a.in.g)[t * a.in.g_stride + head];
            bin[i] = static_cast<const T*>(a.in.beta)[t * a.in.beta_stride + head];
        }

    // K and Q: a warp takes eight rows at a time, lane = row + 8 * column
    // group, so that a store of 8 lanes fills one 8x8 block.  Raw elements go to
    // where their planes will be, all of them asked for at once; while they
    // come, the decays are added up.  Rows and columns that are not there are
    // zero.
    uint8_t* keys = a.keys + (slot * hk + khead) * KeyImage::bytes(DK, NT);
    const bool leave = head % group == 0;
    const int r = lane & 7, c4 = lane >> 3;
    const uint32_t sm = umma::smem_u32(smem);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const int rg = warp * 2 + (w & 1), row = rg * 8 + r;
        const bool isq = w >= 2;
        const int64_t t = tok + min(row, rows - 1);
        const T* p = isq ? static_cast<const T*>(a.in.q) + t * a.in.q_stride + (int64_t)khead * dk
                         : static_cast<const T*>(a.in.k) + t * a.in.k_stride + (int64_t)khead * dk;
#pragma unroll
        for (int i = 0; i < CG / 4; ++i) {
            const int col = (c4 + 4 * i) * 8;
            const bool in = row < rows && col < dk;
            const uint32_t to = sm + (isq ? 0 : kKey) + (rg * CG + c4 + 4 * i) * kTile + r * 16;
#pragma unroll
            for (int n = 0; n < NT; ++n) cp16(to + n * 2 * kKey, p + (in ? col + n * (16 / (int)sizeof(T)) : 0), in);
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    // Running sums of the log decays.
    Two G[2];
    float gam[2], rest[2], most = 1.0f, p_unit = 1.0f / kPScale;
    if (adds) {
        Two g[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float x = 2 * lane + i < rows ? to_f(gin[i]) : 0.0f;
            g[i] = two_log2(x < kMinLogDecay ? kMinLogDecay : x);      // a NaN stays
        }
        Two sum = two_add(g[0], g[1]);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const Two up = {__shfl_up_sync(0xffffffffu, sum.h, o), __shfl_up_sync(0xffffffffu, sum.l, o)};
            const Two both = two_add(up, sum);
            if (lane >= o) sum = both;
        }
        const Two total = {__shfl_sync(0xffffffffu, sum.h, 31), __shfl_sync(0xffffffffu, sum.l, 31)};
        Two before = {__shfl_up_sync(0xffffffffu, sum.h, 1), __shfl_up_sync(0xffffffffu, sum.l, 1)};
        if (lane == 0) before = {0.0f, 0.0f};
        G[0] = two_add(before, g[0]);
        G[1] = sum;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            gam[i] = exp2f(G[i].h + G[i].l);
            rest[i] = exp2f((total.h - G[i].h) + (total.l - G[i].l));
            most = fmaxf(most, rest[i]);
        }
        most = warp_max(most);
        if (__any_sync(0xffffffffu, g[0].h > 0.0f || g[1].h > 0.0f)) {
            // States may grow.  Of the decays D_ij, j <= i, the largest is
            // that of the largest rise of G: P is divided by a power of two no
            // smaller than it.  (Without growth D is at most 1, and P's unit
            // does not depend on the decays.)
            float low = fminf(G[0].h, G[1].h);      // of this lane's tokens and those before
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float up = __shfl_up_sync(0xffffffffu, low, o);
                if (lane >= o) low = fminf(low, up);
            }
            const float below = __shfl_up_sync(0xffffffffu, low, 1);      // of the lanes before
            float rise = fmaxf(G[1].h - G[0].h, 0.0f);
            if (lane > 0) rise = fmaxf(rise, fmaxf(G[0].h, G[1].h) - below);
            p_unit *= __uint_as_float((uint32_t)(127 + (int)ceilf(fminf(warp_max(rise), 120.0f))) << 23);
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");      // a lane reads its own copies only
#pragma unroll 1
    for (int w = 0; w < 4; ++w) {
        const int rg = warp * 2 + (w & 1);
        const bool isq = w >= 2;
        uint8_t* to = smem + (isq ? 0 : kKey) + (rg * CG + c4) * kTile + r * 16;
        Raw<T> raw[CG / 4];
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < CG / 4; ++i) {
            raw[i].load(to + 4 * i * kTile, 2 * kKey);
            float x[8];
            raw[i].get(x);
#pragma unroll
            for (int z = 0; z < 8; ++z) m = fmaxf(m, fabsf(x[z]));
        }
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
        const float unit = row_unit(m, isq ? 126 : 60), inv = pow2_inv(unit);
        if (c4 == 0) (isq ? kqv : kap)[rg * 8 + r] = unit;
#pragma unroll
        for (int i = 0; i < CG / 4; ++i) {
            float x[8];
            raw[i].get(x);
            uint32_t pl[4][NT];
#pragma unroll
            for (int z = 0; z < 4; ++z) planes_h<NT>(x[2 * z] * inv, x[2 * z + 1] * inv, pl[z]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint4 v = make_uint4(pl[0][n], pl[1][n], pl[2][n], pl[3][n]);
                *reinterpret_cast<uint4*>(to + 4 * i * kTile + n * 2 * kKey) = v;
                if (leave)
                    *reinterpret_cast<uint4*>(keys + (isq ? NT * kKey : 0) + n * kKey + (rg * CG + c4 + 4 * i) * kTile + r * 16) = v;
            }
        }
    }
    umma::fence_smem_to_async();
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = s_tmem;
    if (threadIdx.x == 0) {
        constexpr uint32_t kId = umma::instr_desc(umma::kTypeF16, false, false, 128, kChunk);
        const uint32_t base = umma::smem_u32(smem);
        bool first = true;
#pragma unroll
        for (int i = NT - 1; i >= 0; --i)      // the small products first: fp32 gradients 6e-7 off, 1.2e-6 in the other order
#pragma unroll
            for (int j = NT - 1; j >= 0; --j)
                if (i + j < NT) {
                    const uint64_t da = umma::smem_desc(base + i * 2 * kKey, kTile, CG * kTile);
                    const uint64_t db = umma::smem_desc(base + j * 2 * kKey + kKey, kTile, CG * kTile);
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        umma::mma_f16(tmem, da + k * (2 * kTile / 16), db + k * (2 * kTile / 16), kId, first ? 0u : 1u);
                        first = false;
                    }
                }
        umma::commit(&bar);
    }
    __syncwarp();
    if (adds) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = 2 * lane + i;
            const float b = t < rows ? to_f(bin[i]) : 0.0f, k = kap[t];
            const float bk = b * k * k, qs = t < rows ? a.in.scale * kqv[t] : 0.0f;
            vec[V_GHI * kChunk + t] = G[i].h;
            vec[V_GLO * kChunk + t] = G[i].l;
            vec[V_GAM * kChunk + t] = gam[i];
            vec[V_REST * kChunk + t] = rest[i];
            vec[V_BETA * kChunk + t] = bk;
            vec[V_KINV * kChunk + t] = pow2_inv(k);
            vec[V_QINV * kChunk + t] = pow2_inv(kqv[t]);
            vec[V_QS * kChunk + t] = qs;
            vec[V_OS * kChunk + t] = qs * gam[i];
            vec[V_DV * kChunk + t] = b * k;
            vec[V_DS * kChunk + t] = bk * gam[i];
            if (t == 0) {
                vec[V_MISC * kChunk + kMost] = most;
                vec[V_MISC * kChunk + kPUnit] = p_unit;
            }
        }
    }
    __syncthreads();      // the vectors are there
    // a wait that gives up leaves this chunk's results wrong, and says so
    if (!umma::mbar_wait(&bar, 0, kWaitNs)) atomicAdd(a.status + OFRL_STAT_TIMEOUT, 1);
    __syncwarp();
    umma::fence_after_sync();
    const int m4 = lane >> 3, r8 = lane & 7;
    uint8_t* pairs = a.pairs + (slot * hv + head) * kPairBytes;
    {
        // Row i of P (warps 0, 1) or of A (2, 3), 16 columns at a time: P to
        // global memory, A's blocks below the diagonal as images, the diagonal
        // block as floats, column by column.  The keys' place is free.
        const float *ghi = vec + V_GHI * kChunk, *glo = vec + V_GLO * kChunk;
        const int i = (warp & 1) * 32 + lane, ib = i >> 4;
        const bool isk = warp >= 2;
        const float gi = ghi[i], li = glo[i], f = isk ? vec[V_BETA * kChunk + i] : pow2_inv(vec[V_MISC * kChunk + kPUnit]);
        const uint32_t row = tmem + ((uint32_t)(warp * 32) << 16);
        const int at = (i >> 3) * 8 * kTile + (i & 7) * 16;      // of column 0 in an image
#pragma unroll 1
        for (int jb = 0; jb < 4; ++jb) {
            if (jb >= 2 && (warp & 1) == 0) {      // rows 0 .. 31 end before
                if (!isk)
#pragma unroll
                    for (int n = 0; n < 2 * NM; ++n)
                        *reinterpret_cast<uint4*>(pairs + kSquare + (n >> 1) * kPairFirst + at + (2 * jb + (n & 1)) * kTile) =
                            make_uint4(0, 0, 0, 0);
                continue;
            }
            float x[16];
            umma::tmem_ld16(row + jb * 16, x);
            umma::tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 16; c += 4) {
                const float4 h4 = *reinterpret_cast<const float4*>(ghi + jb * 16 + c);
                const float4 l4 = *reinterpret_cast<const float4*>(glo + jb * 16 + c);
                const float gh[4] = {h4.x, h4.y, h4.z, h4.w}, gl[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const int j = jb * 16 + c + z;
                    const float y = x[c + z] * f * exp_2<NM>((gi - gh[z]) + (li - gl[z]));
                    x[c + z] = j < i + (isk ? 0 : 1) ? y : 0.0f;
                }
            }
            if (!isk) {
#pragma unroll
                for (int c = 0; c < 16; c += 8) {
                    uint32_t pl[4][NM];
#pragma unroll
                    for (int z = 0; z < 4; ++z) planes_h<NM>(x[c + 2 * z], x[c + 2 * z + 1], pl[z]);
#pragma unroll
                    for (int n = 0; n < NM; ++n)
                        *reinterpret_cast<uint4*>(pairs + kSquare + n * kPairFirst + at + (2 * jb + c / 8) * kTile) =
                            make_uint4(pl[0][n], pl[1][n], pl[2][n], pl[3][n]);
                }
            } else if (jb < ib) {
#pragma unroll
                for (int c = 0; c < 16; c += 8) {
                    uint32_t pl[4][NB];
#pragma unroll
                    for (int z = 0; z < 4; ++z) planes_b<NB>(x[c + 2 * z], x[c + 2 * z + 1], pl[z]);
#pragma unroll
                    for (int n = 0; n < NB; ++n)
                        *reinterpret_cast<uint4*>(aimg + n * kSquare + at + (2 * jb + c / 8) * kTile) =
                            make_uint4(pl[0][n], pl[1][n], pl[2][n], pl[3][n]);
                }
            } else if (jb == ib) {
#pragma unroll
                for (int c = 0; c < 16; ++c) diag[(ib * 16 + c) * kPitch + (i & 15)] = x[c];      // [j][i]
            }
            __syncwarp();
        }
    }
    umma::fence_before_sync();
    __syncthreads();
    const uint32_t ab = umma::smem_u32(aimg);
    if (inverts) {
        // column c of the inverse: when x_j is known, it leaves every later row
        const int c = lane & 15, w = 2 * (warp & 1) + (lane >> 4);
        const float* D = diag + w * 16 * kPitch;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = i == c ? 1.0f : 0.0f;
#pragma unroll
        for (int j = 0; j < 15; ++j)
#pragma unroll
            for (int q = (j + 1) / 4; q < 4; ++q) {
                const float4 aj = *reinterpret_cast<const float4*>(D + j * kPitch + 4 * q);
                const float av[4] = {aj.x, aj.y, aj.z, aj.w};
#pragma unroll
                for (int z = 0; z < 4; ++z)
                    if (4 * q + z > j) x[4 * q + z] = fmaf(-av[z], x[j], x[4 * q + z]);
            }
        // row c of T_ww^T
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t pl[4][NB];
#pragma unroll
            for (int z = 0; z < 4; ++z) planes_b<NB>(x[8 * h + 2 * z], x[8 * h + 2 * z + 1], pl[z]);
#pragma unroll
            for (int n = 0; n < NB; ++n)
                *reinterpret_cast<uint4*>(aimg + n * kSquare + ((2 * w + (c >> 3)) * 8 + 2 * w + h) * kTile + (c & 7) * 16) =
                    make_uint4(pl[0][n], pl[1][n], pl[2][n], pl[3][n]);
        }
    }
    __syncthreads();
    // block (row block, column block) of the image as a fragment
    auto block = [&](uint32_t (&f)[NB][4], int rb, int cb, bool rows_first) {
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const int hi = m4 >> 1, lo = m4 & 1;
            ldsm4(f[n], ab + n * kSquare + ((2 * rb + (rows_first ? lo : hi)) * 8 + 2 * cb + (rows_first ? hi : lo)) * kTile + r8 * 16);
        }
    };
#pragma unroll 1
    for (int r = warp + 1; r < 4; ++r) {
        float z[2][4];
        zero(z);
#pragma unroll 1
        for (int t = warp; t < r; ++t) {
            uint32_t ft[NB][4], fa[NB][4];
            block(ft, warp, t, true);        // T_tw^T, an A operand
            block(fa, r, t, false);          // A_rt, [n][k]
#pragma unroll
            for (int i = NB - 1; i >= 0; --i)
#pragma unroll
                for (int j = NB - 1; j >= 0; --j)
                    if (i + j < NB) {
                        mma_b(z[0], ft[i], fa[j][0], fa[j][1]);
                        mma_b(z[1], ft[i], fa[j][2], fa[j][3]);
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
        float tb[2][4];
        zero(tb);
#pragma unroll
        for (int j = NB - 1; j >= 0; --j) {
            uint32_t f[4];      // T_rr^T is stored [k][n]
            ldsm4t(f, ab + j * kSquare + ((2 * r + (m4 & 1)) * 8 + 2 * r + (m4 >> 1)) * kTile + r8 * 16);
#pragma unroll
            for (int i = NB - 1; i >= 0; --i)
                if (i + j < NB) {
                    mma_b(tb[0], zp[i], f[0], f[1]);
                    mma_b(tb[1], zp[i], f[2], f[3]);
                }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t pl[NB];
                planes_b<NB>(tb[t][2 * h], tb[t][2 * h + 1], pl);
#pragma unroll
                for (int n = 0; n < NB; ++n)
                    *reinterpret_cast<uint32_t*>(aimg + n * kSquare + ((2 * warp + h) * 8 + 2 * r + t) * kTile + lane * 4) = pl[n];
            }
        __syncwarp();
    }
    // block row `warp` of T^T to global memory, with its power of two: a lane
    // takes eight columns of a row, four times
    float t_most = 0.0f;
    {
        float x[4][8];
        float mx = 0.0f;
        const int row = lane & 15;
        const int at = ((2 * warp + (row >> 3)) * 8) * kTile + (row & 7) * 16;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int cg = 2 * k + (lane >> 4);
#pragma unroll
            for (int z = 0; z < 8; ++z) x[k][z] = 0.0f;
            if (k >= warp)
#pragma unroll
                for (int n = NB - 1; n >= 0; --n) {
                    const uint4 v = *reinterpret_cast<const uint4*>(aimg + n * kSquare + at + cg * kTile);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const float2 f = unpack_b(w[z]);
                        x[k][2 * z] += f.x;
                        x[k][2 * z + 1] += f.y;
                    }
                }
#pragma unroll
            for (int z = 0; z < 8; ++z) mx = fmaxf(mx, fabsf(x[k][z]));
        }
        t_most = warp_max(mx);
        const float up = scale_up(t_most);
        if (lane < 16) {
            const int j = warp * 16 + lane;
            const float inv = pow2_inv(up);
            vec[V_TINV * kChunk + j] = inv;
            vec[V_XV * kChunk + j] = vec[V_DV * kChunk + j] * inv;
            vec[V_XS * kChunk + j] = vec[V_DS * kChunk + j] * inv;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t pl[4][NM];
#pragma unroll
            for (int z = 0; z < 4; ++z) planes_h<NM>(x[k][2 * z] * up, x[k][2 * z + 1] * up, pl[z]);
#pragma unroll
            for (int n = 0; n < NM; ++n)
                *reinterpret_cast<uint4*>(pairs + n * kPairFirst + at + (2 * k + (lane >> 4)) * kTile) =
                    make_uint4(pl[0][n], pl[1][n], pl[2][n], pl[3][n]);
        }
    }
    // A chunk within which states grow, by g or by beta |k|^2 above two, beyond what
    // operands under one power of two hold: x becomes NaN, which makes the chain go
    // over the episode token by token (delta_redo.cuh).  Gradients have no such
    // way: beyond their limit, scale kq becomes NaN and with it the gradients of
    // this chunk and those before it.  Outputs of a chunk's first tokens were 3e-5
    // of their size off after growth of 2^18 in fp32 and 1e-2 after 2^28 in bf16,
    // gradients 8e-7 and 3.6e-4 (fp32) and 1.7e-3 both times, all of them wrong
    // after 2^37.
    constexpr float kReads = NM == 2 ? 0x1p16f : 0x1p24f, kLearns = sizeof(T) == 4 ? 0x1p20f : 0x1p24f;
    const float grows = fmaxf(t_most, vec[V_MISC * kChunk + kPUnit] * kPScale);
    if (__syncthreads_or(grows > kReads)) {
        const bool learns = !__syncthreads_or(grows > kLearns);
        if (threadIdx.x < kChunk) {
            vec[V_XV * kChunk + threadIdx.x] = NAN;
            if (!learns) vec[V_QS * kChunk + threadIdx.x] = NAN;
        }
        __syncthreads();
    }
    for (int i = threadIdx.x; i < kVecBytes / 16; i += kPrepThreads)
        reinterpret_cast<uint4*>(pairs + 2 * kSquare)[i] = reinterpret_cast<const uint4*>(vec)[i];
    umma::fence_after_sync();
    if (warp == 3) {
        umma::mbar_wait(&bar, 0, kWaitNs);      // a product that was given up on may still write
        umma::tmem_dealloc(tmem, kChunk);
    }
}

template <typename T, int DK, int NM>
cudaError_t run(const PrepArgs& p, int64_t grid, cudaStream_t st) {
    constexpr int smem = PrepShared<T, DK, NM>::kBytes;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = opt_in(delta_prep_kernel<T, DK, NM>, smem, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(delta_prep_kernel<T, DK, NM>, dim3((unsigned)grid), dim3(kPrepThreads), smem, st, p);
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
    const int64_t grid = slots_of(a.in.tokens, a.episodes) * a.shape.v_heads;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    const bool wide = a.shape.k_dim > 64;
    if (a.shape.dtype == OFRL_DTYPE_F32) return wide ? run<float, 128, 2>(p, grid, st) : run<float, 64, 2>(p, grid, st);
    if (planes == 2)
        return wide ? run<__nv_bfloat16, 128, 2>(p, grid, st) : run<__nv_bfloat16, 64, 2>(p, grid, st);
    return wide ? run<__nv_bfloat16, 128, 1>(p, grid, st) : run<__nv_bfloat16, 64, 1>(p, grid, st);
}

}  // namespace delta
}  // namespace ofrl
