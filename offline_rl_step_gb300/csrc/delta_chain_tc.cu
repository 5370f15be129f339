// The two passes over an episode's chunks in order, for bf16 tokens and more
// than 64 value channels, on tcgen05 (delta_chain.cu has the formulas and the
// passes for everything else).
//
// The value channels are the 128 accumulator rows, so a thread has a row: no
// value passes between threads but the largest magnitude of a saved image.
// One warpgroup ("tokens") turns the products over a chunk's tokens into the
// next one's operand, the other ("state") keeps the state's rows in its
// registers and makes them an operand; operands go through shared memory,
// where they also are the images the backward pass wants.  Per chunk,
// forward:
//   X = S [K; Q]^T -> x -> U = x T^T -> dS = (rest U) K -> S     (the chain)
//                                    -> O2 = U P^T -> outputs    (beside it)
// About 3.5 us a chunk of 128 x 128 go down to the latency of three products
// and three conversions; mma.sync with 16 rows a warp reads every operand
// eight times from shared memory instead.

#include "delta_mma.cuh"

namespace ofrl {
namespace delta {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 128;                       // accumulator rows: value channels
constexpr int kCol = (kRows / 8) * kTile;        // bytes of a column group of an operand image
constexpr int kTok = kRows * kChunk * 2;         // [rows][64 tokens] image
constexpr uint64_t kWaitNs = 1000000000ull;

struct TcArgs {
    ofrl_delta_shape shape;
    ofrl_delta_tokens in;
    const int32_t* ends;
    const uint8_t* keys;
    const uint8_t* pairs;
    const float* first;
    float* last;
    __nv_bfloat16* out;
    int64_t out_stride;
    const __nv_bfloat16* rows;
    int64_t row_stride;
    uint8_t* state_img;
    uint8_t* vec_img;
    float* state_unit;
    float* vec_unit;
    unsigned* counter;
    int32_t* status;
};

template <int DK>
struct Smem {
    static constexpr int kKey = kChunk * DK * 2;
    static constexpr int kState = kRows * DK * 2;
    static constexpr int kStage = 2 * kKey + (int)kPairFirst;
    static constexpr int off_s = 0;                      // the state as an operand
    static constexpr int off_a = off_s + kState;         // forward: x; backward: dO
    static constexpr int off_b = off_a + kTok;           // forward: U; backward: dU, then R
    static constexpr int off_c = off_b + kTok;           // forward: rest U; backward: gamma dO
    static constexpr int off_d = off_c + kTok;           // backward: -gamma dv
    static constexpr int off_stage = off_d + kTok;
    static constexpr int off_row = off_stage + 2 * kStage;      // per row: powers of two
    static constexpr int kBytes = off_row + 4 * kRows * 4;
    static_assert(kBytes <= 226 * 1024, "shared memory");
};

struct Bars {
    uint64_t full[2], empty[2];
    uint64_t s_ready, o_done, u_ready;      // between the warpgroups
    uint64_t a, b, t, s, p;                 // products done
    int dead;
    uint32_t tmem;
    float most[2][4];
};

template <int BAR>
__device__ __forceinline__ void group_sync() {
    asm volatile("bar.sync %0, 128;" ::"n"(BAR) : "memory");
}

// Wait of a whole warp; once one has given up, none waits and the pass runs on
// over what is there (warps that meet at barriers all get there).
__device__ __forceinline__ void wait(Bars& b, uint64_t* bar, int turn) {
    if (!*(volatile int*)&b.dead && !umma::mbar_wait(bar, (uint32_t)turn & 1u, kWaitNs)) b.dead = 1;
    __syncwarp();
    umma::fence_after_sync();
}

// N columns of this thread's row.
template <int N>
__device__ __forceinline__ void tmem_row(uint32_t taddr, float (&v)[N]) {
#pragma unroll
    for (int c = 0; c < N; c += 16) umma::tmem_ld16(taddr + c, *reinterpret_cast<float(*)[16]>(v + c));
    umma::tmem_ld_wait();
}

__device__ __forceinline__ void mma_run(uint32_t d, uint64_t a, uint32_t a_step, uint64_t b, uint32_t b_step, uint32_t id,
                                        int steps) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < steps) umma::mma_f16(d, a + (uint64_t)k * (a_step >> 4), b + (uint64_t)k * (b_step >> 4), id, k > 0 ? 1u : 0u);
}

// x[0 .. 63] times f as the row of a [rows][64] operand image.
__device__ __forceinline__ void put_row(uint8_t* img, int row, const float (&x)[64], float f) {
    uint8_t* to = img + (row >> 3) * kTile + (row & 7) * 16;
#pragma unroll
    for (int c = 0; c < 64; c += 8)
        *reinterpret_cast<uint4*>(to + c / 8 * kCol) =
            make_uint4(pack_h(x[c] * f, x[c + 1] * f), pack_h(x[c + 2] * f, x[c + 3] * f), pack_h(x[c + 4] * f, x[c + 5] * f),
                       pack_h(x[c + 6] * f, x[c + 7] * f));
}
template <int N>
__device__ __forceinline__ float row_max(const float (&x)[N]) {
    float m[4] = {0, 0, 0, 0};
#pragma unroll
    for (int c = 0; c < N; ++c) m[c & 3] = fmaxf(m[c & 3], fabsf(x[c]));
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// Largest of a warpgroup's values.
template <int BAR>
__device__ __forceinline__ float group_max(float (&most)[4], float v) {
    v = warp_max(v);
    if ((threadIdx.x & 31) == 0) most[(threadIdx.x >> 5) & 3] = v;
    group_sync<BAR>();
    return fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
}

struct Episode {
    int head, khead, chunks;
    Span sp;
    int64_t slot0, states;
};
__device__ __forceinline__ Episode episode(const TcArgs& a) {
    Episode w;
    const int hv = a.shape.v_heads, e = blockIdx.x / hv;
    w.head = blockIdx.x % hv;
    w.khead = w.head / (hv / a.shape.k_heads);
    w.sp = span_of(a.ends, e, (int32_t)a.in.tokens);
    w.chunks = (w.sp.len + kChunk - 1) / kChunk;
    w.slot0 = w.sp.start / kChunk + e;
    w.states = ((int64_t)e * hv + w.head) * a.shape.v_dim * a.shape.k_dim;
    return w;
}

template <int DK>
__device__ __forceinline__ void copy_stage(const TcArgs& a, const Episode& w, uint8_t* smem, Bars& b, int n, int c) {
    using S = Smem<DK>;
    const int64_t slot = w.slot0 + c;
    uint8_t* to = smem + S::off_stage + (n & 1) * S::kStage;
    umma::mbar_expect_tx(&b.full[n & 1], S::kStage);
    umma::bulk_g2s(to, a.keys + (slot * a.shape.k_heads + w.khead) * KeyImage::bytes(DK, 1), 2 * S::kKey, &b.full[n & 1]);
    umma::bulk_g2s(to + 2 * S::kKey, a.pairs + (slot * a.shape.v_heads + w.head) * kPairBytes, (uint32_t)kPairFirst,
                   &b.full[n & 1]);
}

// Channel `row` of a chunk's tokens; zero past their end and past v_dim.
__device__ __forceinline__ void load_tokens(const TcArgs& a, const Episode& w, int c, int row, uint16_t (&x)[64]) {
    const int rows = w.sp.len - c * kChunk;
    const uint16_t* p = reinterpret_cast<const uint16_t*>(a.rows) + ((int64_t)w.sp.start + c * kChunk) * a.row_stride +
                        (int64_t)w.head * a.shape.v_dim + row;
    const bool on = row < a.shape.v_dim && c >= 0 && c < w.chunks;
#pragma unroll
    for (int i = 0; i < 64; ++i) x[i] = on && i < rows ? p[i * a.row_stride] : (uint16_t)0;
}
__device__ __forceinline__ float widen(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }

__device__ __forceinline__ void store_tokens(const TcArgs& a, const Episode& w, int c, int row, const float (&x)[64]) {
    if (row >= a.shape.v_dim) return;
    const int rows = w.sp.len - c * kChunk;
    __nv_bfloat16* p = a.out + ((int64_t)w.sp.start + c * kChunk) * a.out_stride + (int64_t)w.head * a.shape.v_dim + row;
#pragma unroll
    for (int i = 0; i < 64; ++i)
        if (i < rows) p[i * a.out_stride] = __float2bfloat16_rn(x[i]);
}

// Four columns' values of a vector.
__device__ __forceinline__ void four(const float* vec, int which, int c, float (&x)[4]) {
    const float4 v = *reinterpret_cast<const float4*>(vec + which * kChunk + c);
    x[0] = v.x;
    x[1] = v.y;
    x[2] = v.z;
    x[3] = v.w;
}

template <int DK>
__device__ __forceinline__ void load_row(const float* from, float (&s)[DK], int row, int dv, int dk) {
#pragma unroll
    for (int c = 0; c < DK; c += 4) {
        float4 v = make_float4(0, 0, 0, 0);
        if (from != nullptr && row < dv && c < dk) v = *reinterpret_cast<const float4*>(from + (int64_t)row * dk + c);
        s[c] = v.x;
        s[c + 1] = v.y;
        s[c + 2] = v.z;
        s[c + 3] = v.w;
    }
}
template <int DK>
__device__ __forceinline__ void put_state(uint8_t* img, int row, const float (&s)[DK], float f) {
    uint8_t* to = img + (row >> 3) * kTile + (row & 7) * 16;
#pragma unroll
    for (int c = 0; c < DK; c += 8)
        *reinterpret_cast<uint4*>(to + c / 8 * kCol) =
            make_uint4(pack_h(s[c] * f, s[c + 1] * f), pack_h(s[c + 2] * f, s[c + 3] * f), pack_h(s[c + 4] * f, s[c + 5] * f),
                       pack_h(s[c + 6] * f, s[c + 7] * f));
}

__device__ __forceinline__ void init_bars(Bars& b) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            umma::mbar_init(&b.full[i], 1);
            umma::mbar_init(&b.empty[i], 8);
        }
        umma::mbar_init(&b.s_ready, 1);
        umma::mbar_init(&b.u_ready, 1);
        umma::mbar_init(&b.o_done, 4);
        umma::mbar_init(&b.a, 1);
        umma::mbar_init(&b.b, 1);
        umma::mbar_init(&b.t, 1);
        umma::mbar_init(&b.s, 1);
        umma::mbar_init(&b.p, 1);
        b.dead = 0;
        umma::fence_mbar_init();
    }
}

// TMEM columns.
constexpr int t_x = 0, t_q = 64, t_u = 128, t_o = 192, t_s = 256, t_s2 = 384;

template <int DK, bool SAVE>
__global__ void __launch_bounds__(kThreads) delta_forward_tc_kernel(const __grid_constant__ TcArgs a) {
    using S = Smem<DK>;
    constexpr int CG = DK / 8, KS = DK / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(16) Bars b;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = threadIdx.x & 127;
    const Episode w = episode(a);
    const int dk = a.shape.k_dim, dv = a.shape.v_dim;
    init_bars(b);
    if (warp == 0) umma::tmem_alloc(&b.tmem, 512);
    float* s_row = reinterpret_cast<float*>(smem + S::off_row);      // 1 / power of two of the state's rows
    float* u_row = s_row + kRows;                                    // of U's
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = b.tmem, mine = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t base = umma::smem_u32(smem);
    auto vec_of = [&](int n) { return reinterpret_cast<const float*>(smem + S::off_stage + (n & 1) * S::kStage + 2 * S::kKey + 2 * kSquare); };
    auto keys_at = [&](int n) { return base + S::off_stage + (n & 1) * S::kStage; };

    if (warp < 4) {
        uint16_t v[64];
        load_tokens(a, w, 0, row, v);
        pdl_wait();
        if (threadIdx.x == 0 && w.chunks > 0) copy_stage<DK>(a, w, smem, b, 0, 0);
        constexpr uint32_t kIdT = umma::instr_desc(umma::kTypeF16, false, true, kRows, kChunk);
        constexpr uint32_t kIdP = umma::instr_desc(umma::kTypeF16, false, false, kRows, kChunk);
        constexpr uint32_t kIdS = umma::instr_desc(umma::kTypeF16, false, true, kRows, DK);
        for (int n = 0; n < w.chunks; ++n) {
            const float* vec = vec_of(n);
            wait(b, &b.full[n & 1], n >> 1);
            wait(b, &b.s_ready, n);
            wait(b, &b.a, n);
            if (threadIdx.x == 0 && n + 1 < w.chunks) {
                if (n > 0 && !b.dead && !umma::mbar_wait(&b.empty[(n + 1) & 1], (uint32_t)((n + 1) / 2 - 1) & 1u, kWaitNs)) b.dead = 1;
                if (!b.dead) copy_stage<DK>(a, w, smem, b, n + 1, n + 1);
            }
            __syncwarp();
            const float s_inv = s_row[row];
            float x[64];
            tmem_row(mine + t_x, x);
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
                float f[4], g[4];
                four(vec, V_XV, c, f);
                four(vec, V_XS, c, g);
#pragma unroll
                for (int z = 0; z < 4; ++z) x[c + z] = f[z] * widen(v[c + z]) - (g[z] * s_inv) * x[c + z];
            }
            const float x_up = scale_up(row_max(x)), x_inv = pow2_inv(x_up);
            put_row(smem + S::off_a, row, x, x_up);
            umma::fence_smem_to_async();
            umma::fence_before_sync();
            group_sync<1>();
            umma::fence_after_sync();
            const uint32_t pair = keys_at(n) + 2 * S::kKey;
            if (threadIdx.x == 0) {
                mma_run(tmem + t_u, umma::smem_desc(base + S::off_a, kCol, kTile), 2 * kCol, umma::smem_desc(pair, 8 * kTile, kTile),
                        2 * 8 * kTile, kIdT, 4);
                umma::commit(&b.t);
                if (SAVE) umma::bulk_wait_read();      // U's image of the chunk before
            }
            load_tokens(a, w, n + 1, row, v);
            __syncwarp();
            if (SAVE) group_sync<1>();
            wait(b, &b.t, n);
            tmem_row(mine + t_u, x);
            float u_max = row_max(x) * x_inv * vec[V_MISC * kChunk];
            if (SAVE) u_max = group_max<1>(b.most[0], u_max);
            const float u_up = scale_up(u_max), u_inv = pow2_inv(u_up), u_f = u_up * x_inv;
            put_row(smem + S::off_b, row, x, u_f);
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
                float f[4];
                four(vec, V_REST, c, f);
#pragma unroll
                for (int z = 0; z < 4; ++z) x[c + z] *= f[z];
            }
            put_row(smem + S::off_c, row, x, u_f);
            u_row[row] = u_inv;
            umma::fence_smem_to_async();
            umma::fence_before_sync();
            group_sync<1>();
            umma::fence_after_sync();
            if (threadIdx.x == 0) {
                umma::mbar_arrive(&b.u_ready);
                mma_run(tmem + t_s, umma::smem_desc(base + S::off_c, kCol, kTile), 2 * kCol,
                        umma::smem_desc(keys_at(n), CG * kTile, kTile), 2 * CG * kTile, kIdS, 4);
                umma::commit(&b.s);
                mma_run(tmem + t_o, umma::smem_desc(base + S::off_b, kCol, kTile), 2 * kCol,
                        umma::smem_desc(pair + kSquare, kTile, 8 * kTile), 2 * kTile, kIdP, 4);
                umma::commit(&b.p);
                if (SAVE) {
                    const int64_t at = (w.slot0 + n) * a.shape.v_heads + w.head;
                    umma::bulk_s2g(a.vec_img + at * kTok, smem + S::off_b, kTok);
                    umma::bulk_commit();
                    a.vec_unit[at] = u_inv;
                }
            }
            __syncwarp();
            wait(b, &b.b, n);
            wait(b, &b.p, n);
            const float p_inv = u_inv * (1.0f / kPScale);
            float o[64];
            tmem_row(mine + t_q, x);
            tmem_row(mine + t_o, o);
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) umma::mbar_arrive(&b.o_done);
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
                float f[4], g[4];
                four(vec, V_OS, c, f);
                four(vec, V_QS, c, g);
#pragma unroll
                for (int z = 0; z < 4; ++z) o[c + z] = (f[z] * s_inv) * x[c + z] + (g[z] * p_inv) * o[c + z];
            }
            __syncwarp();
            if (lane == 0) umma::mbar_arrive(&b.empty[n & 1]);
            store_tokens(a, w, n, row, o);
        }
        if (SAVE && threadIdx.x == 0) umma::bulk_wait_read();
    } else {
        float s[DK];
        load_row(a.first ? a.first + w.states : nullptr, s, row, dv, dk);
        pdl_wait();
        constexpr uint32_t kIdA = umma::instr_desc(umma::kTypeF16, false, false, kRows, kChunk);
        for (int n = 0; n < w.chunks; ++n) {
            if (n > 0) wait(b, &b.b, n - 1);      // what read the image is done
            float most = row_max(s);
            if (SAVE) {
                if (threadIdx.x == 128) umma::bulk_wait_read();      // the image of the chunk before
                most = group_max<2>(b.most[1], most);
            }
            const float up = scale_up(most), inv = pow2_inv(up);
            put_state(smem + S::off_s, row, s, up);
            s_row[row] = inv;
            umma::fence_smem_to_async();
            umma::fence_before_sync();
            group_sync<2>();
            umma::fence_after_sync();
            wait(b, &b.full[n & 1], n >> 1);
            if (n > 0) wait(b, &b.o_done, n - 1);
            if (threadIdx.x == 128) {
                umma::mbar_arrive(&b.s_ready);
                const uint64_t sd = umma::smem_desc(base + S::off_s, kCol, kTile);
                mma_run(tmem + t_x, sd, 2 * kCol, umma::smem_desc(keys_at(n), kTile, CG * kTile), 2 * kTile, kIdA, KS);
                umma::commit(&b.a);
                mma_run(tmem + t_q, sd, 2 * kCol, umma::smem_desc(keys_at(n) + S::kKey, kTile, CG * kTile), 2 * kTile, kIdA, KS);
                umma::commit(&b.b);
                if (SAVE) {
                    const int64_t at = (w.slot0 + n) * a.shape.v_heads + w.head;
                    umma::bulk_s2g(a.state_img + at * S::kState, smem + S::off_s, S::kState);
                    umma::bulk_commit();
                    a.state_unit[at] = inv;
                }
            }
            __syncwarp();
            const float keep = vec_of(n)[V_GAM * kChunk + kChunk - 1];
            wait(b, &b.u_ready, n);
            wait(b, &b.s, n);
            const float u_inv = u_row[row];
#pragma unroll
            for (int c = 0; c < DK; c += 32) {
                float d[32];
                tmem_row(mine + t_s + c, d);
#pragma unroll
                for (int z = 0; z < 32; ++z) s[c + z] = keep * s[c + z] + u_inv * d[z];
            }
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) umma::mbar_arrive(&b.empty[n & 1]);
        }
        if (SAVE && threadIdx.x == 128) umma::bulk_wait_read();
    }
    __syncthreads();
    umma::fence_after_sync();
    if (threadIdx.x == 0 && b.dead) atomicAdd(a.status + OFRL_STAT_TIMEOUT, 1);
    if (warp == 0) umma::tmem_dealloc(tmem, 512);
}

template <int DK>
__global__ void __launch_bounds__(kThreads) delta_reverse_tc_kernel(const __grid_constant__ TcArgs a) {
    using S = Smem<DK>;
    constexpr int CG = DK / 8, KS = DK / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(16) Bars b;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = threadIdx.x & 127;
    const Episode w = episode(a);
    const int dk = a.shape.k_dim, dv = a.shape.v_dim;
    pdl_trigger();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.counter = 0;
    init_bars(b);
    if (warp == 0) umma::tmem_alloc(&b.tmem, 512);
    float* s_row = reinterpret_cast<float*>(smem + S::off_row);      // 1 / power of two of the state's rows
    float* o_row = s_row + kRows;                                    // of gamma dO's, for two chunks
    float* r_row = o_row + 2 * kRows;                                // of gamma dv's
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = b.tmem, mine = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t base = umma::smem_u32(smem);
    auto vec_of = [&](int n) { return reinterpret_cast<const float*>(smem + S::off_stage + (n & 1) * S::kStage + 2 * S::kKey + 2 * kSquare); };
    auto keys_at = [&](int n) { return base + S::off_stage + (n & 1) * S::kStage; };

    if (warp < 4) {
        uint16_t v[64];
        load_tokens(a, w, w.chunks - 1, row, v);
        if (threadIdx.x == 0 && w.chunks > 0) copy_stage<DK>(a, w, smem, b, 0, w.chunks - 1);
        constexpr uint32_t kIdP = umma::instr_desc(umma::kTypeF16, false, true, kRows, kChunk);
        constexpr uint32_t kIdT = umma::instr_desc(umma::kTypeF16, false, false, kRows, kChunk);
        constexpr uint32_t kIdS = umma::instr_desc(umma::kTypeF16, false, true, kRows, DK);
        for (int n = 0; n < w.chunks; ++n) {
            const int c0 = w.chunks - 1 - n;
            const float* vec = vec_of(n);
            const uint32_t pair = keys_at(n) + 2 * S::kKey;
            wait(b, &b.full[n & 1], n >> 1);
            if (n > 0) wait(b, &b.s, n - 1);      // what read the images below is done
            // dO scale kq, for P; and times gamma, for the state
            float x[64], y[64];
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
                float f[4], g[4];
                four(vec, V_QS, c, f);
                four(vec, V_GAM, c, g);
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    x[c + z] = widen(v[c + z]) * f[z];
                    y[c + z] = x[c + z] * g[z];
                }
            }
            const float a_up = scale_up(row_max(x)), a_inv = pow2_inv(a_up);
            put_row(smem + S::off_a, row, x, a_up);
            const float o_up = scale_up(row_max(y));
            put_row(smem + S::off_c, row, y, o_up);
            o_row[(n & 1) * kRows + row] = pow2_inv(o_up);
            if (threadIdx.x == 0) umma::bulk_wait_read();      // R's image of the chunk before
            umma::fence_smem_to_async();
            umma::fence_before_sync();
            group_sync<1>();
            umma::fence_after_sync();
            if (threadIdx.x == 0) {
                mma_run(tmem + t_q, umma::smem_desc(base + S::off_a, kCol, kTile), 2 * kCol,
                        umma::smem_desc(pair + kSquare, 8 * kTile, kTile), 2 * 8 * kTile, kIdP, 4);
                umma::commit(&b.b);
            }
            __syncwarp();
            wait(b, &b.b, n);
            tmem_row(mine + t_q, y);
            wait(b, &b.s_ready, n);
            wait(b, &b.a, n);
            if (threadIdx.x == 0 && n + 1 < w.chunks) {
                if (n > 0 && !b.dead && !umma::mbar_wait(&b.empty[(n + 1) & 1], (uint32_t)((n + 1) / 2 - 1) & 1u, kWaitNs)) b.dead = 1;
                if (!b.dead) copy_stage<DK>(a, w, smem, b, n + 1, w.chunks - 2 - n);
            }
            __syncwarp();
            const float s_inv = s_row[row], p_inv = a_inv * (1.0f / kPScale);
            tmem_row(mine + t_x, x);
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
                float f[4];
                four(vec, V_REST, c, f);
#pragma unroll
                for (int z = 0; z < 4; ++z) x[c + z] = (f[z] * s_inv) * x[c + z] + p_inv * y[c + z];
            }
            const float u_up = scale_up(row_max(x)), u_inv = pow2_inv(u_up);
            put_row(smem + S::off_b, row, x, u_up);
            umma::fence_smem_to_async();
            umma::fence_before_sync();
            group_sync<1>();
            umma::fence_after_sync();
            if (threadIdx.x == 0) {
                mma_run(tmem + t_u, umma::smem_desc(base + S::off_b, kCol, kTile), 2 * kCol, umma::smem_desc(pair, kTile, 8 * kTile),
                        2 * kTile, kIdT, 4);
                umma::commit(&b.t);
            }
            __syncwarp();
            load_tokens(a, w, c0 - 1, row, v);
            wait(b, &b.t, n);
            tmem_row(mine + t_u, x);
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
                float f[4], g[4];
                four(vec, V_TINV, c, f);
                four(vec, V_DS, c, g);
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    x[c + z] *= f[z] * u_inv;
                    y[c + z] = -x[c + z] * g[z];
                }
            }
            const float r_up = scale_up(row_max(y));
            put_row(smem + S::off_d, row, y, r_up);
            r_row[row] = pow2_inv(r_up);
            const float i_up = scale_up(group_max<1>(b.most[0], row_max(x)));
            put_row(smem + S::off_b, row, x, i_up);
            umma::fence_smem_to_async();
            umma::fence_before_sync();
            group_sync<1>();
            umma::fence_after_sync();
            if (threadIdx.x == 0) {
                umma::mbar_arrive(&b.u_ready);
                mma_run(tmem + t_s, umma::smem_desc(base + S::off_c, kCol, kTile), 2 * kCol,
                        umma::smem_desc(keys_at(n) + S::kKey, CG * kTile, kTile), 2 * CG * kTile, kIdS, 4);
                mma_run(tmem + t_s2, umma::smem_desc(base + S::off_d, kCol, kTile), 2 * kCol,
                        umma::smem_desc(keys_at(n), CG * kTile, kTile), 2 * CG * kTile, kIdS, 4);
                umma::commit(&b.s);
                const int64_t at = (w.slot0 + c0) * a.shape.v_heads + w.head;
                umma::bulk_s2g(a.vec_img + at * kTok, smem + S::off_b, kTok);
                umma::bulk_commit();
                a.vec_unit[at] = pow2_inv(i_up);
            }
            __syncwarp();
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
                float f[4];
                four(vec, V_DV, c, f);
#pragma unroll
                for (int z = 0; z < 4; ++z) x[c + z] *= f[z];
            }
            __syncwarp();
            if (lane == 0) umma::mbar_arrive(&b.empty[n & 1]);
            store_tokens(a, w, c0, row, x);
        }
        if (threadIdx.x == 0) umma::bulk_wait_read();
    } else {
        float s[DK];
        load_row(a.first ? a.first + w.states : nullptr, s, row, dv, dk);
        constexpr uint32_t kIdA = umma::instr_desc(umma::kTypeF16, false, false, kRows, kChunk);
        for (int n = 0; n < w.chunks; ++n) {
            const int c0 = w.chunks - 1 - n;
            if (threadIdx.x == 128) umma::bulk_wait_read();      // the image of the chunk before
            const float up = scale_up(group_max<2>(b.most[1], row_max(s))), inv = pow2_inv(up);
            put_state(smem + S::off_s, row, s, up);
            s_row[row] = inv;
            umma::fence_smem_to_async();
            umma::fence_before_sync();
            group_sync<2>();
            umma::fence_after_sync();
            wait(b, &b.full[n & 1], n >> 1);
            if (threadIdx.x == 128) {
                umma::mbar_arrive(&b.s_ready);
                mma_run(tmem + t_x, umma::smem_desc(base + S::off_s, kCol, kTile), 2 * kCol,
                        umma::smem_desc(keys_at(n), kTile, CG * kTile), 2 * kTile, kIdA, KS);
                umma::commit(&b.a);
                const int64_t at = (w.slot0 + c0) * a.shape.v_heads + w.head;
                umma::bulk_s2g(a.state_img + at * S::kState, smem + S::off_s, S::kState);
                umma::bulk_commit();
                a.state_unit[at] = inv;
            }
            __syncwarp();
            const float keep = vec_of(n)[V_GAM * kChunk + kChunk - 1];
            wait(b, &b.u_ready, n);
            wait(b, &b.s, n);
            const float o_inv = o_row[(n & 1) * kRows + row], r_inv = r_row[row];
#pragma unroll
            for (int c = 0; c < DK; c += 32) {
                float d[32], e[32];
                tmem_row(mine + t_s + c, d);
                tmem_row(mine + t_s2 + c, e);
#pragma unroll
                for (int z = 0; z < 32; ++z) s[c + z] = keep * s[c + z] + (o_inv * d[z] + r_inv * e[z]);
            }
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) umma::mbar_arrive(&b.empty[n & 1]);
        }
        if (threadIdx.x == 128) umma::bulk_wait_read();
        if (a.last && row < dv) {
            float* to = a.last + w.states + (int64_t)row * dk;
#pragma unroll
            for (int c = 0; c < DK; c += 4)
                if (c < dk) *reinterpret_cast<float4*>(to + c) = make_float4(s[c], s[c + 1], s[c + 2], s[c + 3]);
        }
    }
    __syncthreads();
    umma::fence_after_sync();
    if (threadIdx.x == 0 && b.dead) atomicAdd(a.status + OFRL_STAT_TIMEOUT, 1);
    if (warp == 0) umma::tmem_dealloc(tmem, 512);
}

template <auto KERNEL, int DK>
cudaError_t go(const TcArgs& c, int64_t grid, bool early, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    const cudaError_t e = opt_in(KERNEL, Smem<DK>::kBytes, done);
    if (e != cudaSuccess) return e;
    if (early) return launch_pdl(KERNEL, dim3((unsigned)grid), dim3(kThreads), Smem<DK>::kBytes, st, c);
    KERNEL<<<(unsigned)grid, kThreads, Smem<DK>::kBytes, st>>>(c);
    return cudaGetLastError();
}

TcArgs base_args(const SeqLaunch& a, const Prepared& p, const Images& img) {
    TcArgs c;
    c.shape = a.shape;
    c.in = a.in;
    c.ends = a.ends;
    c.keys = p.keys;
    c.pairs = p.pairs;
    c.state_img = img.state;
    c.vec_img = img.vec;
    c.state_unit = img.state_unit;
    c.vec_unit = img.vec_unit;
    c.counter = a.counter;
    c.status = a.status;
    return c;
}

}  // namespace

cudaError_t launch_chain_forward_tc(const SeqLaunch& a, const Prepared& p, const Images& img, cudaStream_t st) {
    TcArgs c = base_args(a, p, img);
    c.first = a.init;
    c.last = nullptr;
    c.out = static_cast<__nv_bfloat16*>(a.out);
    c.out_stride = (int64_t)a.shape.v_heads * a.shape.v_dim;
    c.rows = static_cast<const __nv_bfloat16*>(a.in.v);
    c.row_stride = a.in.v_stride;
    const int64_t grid = (int64_t)a.episodes * a.shape.v_heads;
    if (a.shape.k_dim > 64)
        return a.saved ? go<delta_forward_tc_kernel<128, true>, 128>(c, grid, true, st)
                       : go<delta_forward_tc_kernel<128, false>, 128>(c, grid, true, st);
    return a.saved ? go<delta_forward_tc_kernel<64, true>, 64>(c, grid, true, st)
                   : go<delta_forward_tc_kernel<64, false>, 64>(c, grid, true, st);
}

cudaError_t launch_chain_reverse_tc(const SeqLaunch& a, const Prepared& p, const Images& img, cudaStream_t st) {
    TcArgs c = base_args(a, p, img);
    c.first = a.d_final;
    c.last = a.d_init;
    c.out = static_cast<__nv_bfloat16*>(a.grads.dv);
    c.out_stride = a.grads.v_stride;
    c.rows = static_cast<const __nv_bfloat16*>(a.dout);
    c.row_stride = (int64_t)a.shape.v_heads * a.shape.v_dim;
    const int64_t grid = (int64_t)a.episodes * a.shape.v_heads;
    return a.shape.k_dim > 64 ? go<delta_reverse_tc_kernel<128>, 128>(c, grid, false, st)
                              : go<delta_reverse_tc_kernel<64>, 64>(c, grid, false, st);
}

}  // namespace delta
}  // namespace ofrl
