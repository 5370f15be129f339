// The two passes over an episode's chunks in order, for bf16 tokens and more
// than 64 value channels, on tcgen05 (delta_chain.cu has the formulas and the
// passes for everything else).
//
// The value channels are the 128 accumulator rows.  Two warpgroups ("tokens")
// turn the products over a chunk's tokens into the next one's operand, two
// ("state") keep the state's rows in their registers and make them an operand;
// a thread has a row and half of the columns.  Operands go through shared
// memory, where they also are the images that the gradients want.  Per chunk:
//   forward   X = S K^T -> x -> U = x T^T -> S += (rest U) K            (the chain)
//             beside it S Q^T, U P^T -> outputs
//   backward  X = dS K^T, dO P -> dU -> R = dU T -> dS -= (gamma dv) K  (the chain)
//             beside it dS += (gamma dO) Q, R -> dv
// What is beside the chain is made by the warps that would wait: outputs and dv
// of a chunk by the state's warps after they have left the next chunk's state,
// dO's operands by the tokens' warps while the state is on its way.
//
// Bound by the chain's latency, three products (0.3 to 0.8 us each with their
// operands' reads) and three conversions: 4 us a chunk of 128 x 128 forward, 5
// back.  About 65k ragged transitions, four heads of 128 x 128: 143 us forward
// (4.1 TB/s in all), 162 us back.  With two warpgroups and every token element
// read and written by itself 219 and 285; with outputs and dv by the tokens'
// warps 164 and 165.

#include "delta_redo.cuh"

namespace ofrl {
namespace delta {
namespace {

constexpr int kThreads = 512;                    // two warpgroups for the tokens, two for the state
constexpr int kTokThreads = 256;
constexpr int kHalf = kChunk / 2;                // tokens of a thread
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
    static constexpr int off_d = off_c + kTok;           // forward: outputs turned around; backward: -gamma dv
    static constexpr int off_stage = off_d + kTok;
    static constexpr int off_turn = off_stage + 2 * kStage;     // a warp's 32 channels x 32 tokens, turned around
    static constexpr int off_row = off_turn + kTok;             // largest magnitudes of halves of rows
    static constexpr int kBytes = off_row + 4 * kRows * 4;
    static_assert(kBytes <= 226 * 1024, "shared memory");
};

struct Bars {
    uint64_t full[2];
    uint64_t s_ready, u_ready;              // from the state's warps, from the tokens'
    uint64_t free;                          // forward: t_q and t_o are read
    uint64_t a, b, t, s, p;              // products done
    uint64_t done[2];                       // after a wait that gave up: everything a thread issued is done
    int dead;
    int copied;                             // chunks whose copies were started
    uint32_t tmem;
    float most[2][8], more[8];
    // 1 / powers of two: the state, U, gamma dO, and what the state takes in (rest U or -gamma dv)
    float s_inv, u_inv, o_inv[2], r_inv;
    alignas(16) float dv_f[2][kChunk];      // backward: factors of dv
};

template <int BAR>
__device__ __forceinline__ void group_sync() {
    asm volatile("bar.sync %0, 256;" ::"n"(BAR) : "memory");
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

// Largest of a row half's magnitudes.
template <int N>
__device__ __forceinline__ float half_max(const float (&x)[N]) {
    float m[4] = {0, 0, 0, 0};
#pragma unroll
    for (int c = 0; c < N; ++c) m[c & 3] = fmaxf(m[c & 3], fabsf(x[c]));
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}
// Largest of the values of all warps that meet here.
__device__ __forceinline__ float all_max(const float (&most)[8]) {
    return fmaxf(fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3])),
                 fmaxf(fmaxf(most[4], most[5]), fmaxf(most[6], most[7])));
}
template <int BAR>
__device__ __forceinline__ float group_max(float (&most)[8], float v) {
    v = warp_max(v);
    if ((threadIdx.x & 31) == 0) most[(threadIdx.x >> 5) & 7] = v;
    group_sync<BAR>();
    return all_max(most);
}
// The same, NaN if one is NaN.
__device__ __forceinline__ float max_nan(float a, float b, float c = 0.0f) {
    float m;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}
template <int N>
__device__ __forceinline__ float half_max_nan(const float (&x)[N]) {
    float m[2] = {0, 0};
#pragma unroll
    for (int c = 0; c < N; c += 4) {
        m[0] = max_nan(m[0], fabsf(x[c]), fabsf(x[c + 1]));
        m[1] = max_nan(m[1], fabsf(x[c + 2]), fabsf(x[c + 3]));
    }
    return max_nan(m[0], m[1]);
}
template <int BAR>
__device__ __forceinline__ float group_max_nan(float (&most)[8], float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    if ((threadIdx.x & 31) == 0) most[(threadIdx.x >> 5) & 7] = v;
    group_sync<BAR>();
    return max_nan(max_nan(max_nan(most[0], most[1], most[2]), most[3], most[4]), max_nan(most[5], most[6], most[7]));
}
// x times f as N columns of a row of an operand image that begins at `to`.
template <int N>
__device__ __forceinline__ void put_cols(uint8_t* to, const float (&x)[N], float f) {
#pragma unroll
    for (int c = 0; c < N; c += 8)
        *reinterpret_cast<uint4*>(to + c / 8 * kCol) =
            make_uint4(pack_h(x[c] * f, x[c + 1] * f), pack_h(x[c + 2] * f, x[c + 3] * f), pack_h(x[c + 4] * f, x[c + 5] * f),
                       pack_h(x[c + 6] * f, x[c + 7] * f));
}

struct Episode {
    int head, khead, chunks;
    Span sp;
    int64_t slot0, states;
};
__device__ __forceinline__ Episode episode(const TcArgs& a, unsigned block) {
    Episode w;
    const int hv = a.shape.v_heads, e = block / hv;
    w.head = block % hv;
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
    b.copied = n + 1;
    uint8_t* to = smem + S::off_stage + (n & 1) * S::kStage;
    umma::mbar_expect_tx(&b.full[n & 1], S::kStage);
    umma::bulk_g2s(to, a.keys + (slot * a.shape.k_heads + w.khead) * KeyImage::bytes(DK, 1), 2 * S::kKey, &b.full[n & 1]);
    umma::bulk_g2s(to + 2 * S::kKey, a.pairs + (slot * a.shape.v_heads + w.head) * kPairBytes, (uint32_t)kPairFirst,
                   &b.full[n & 1]);
}

// A warp's 32 tokens of 32 channels pass through shared memory to be turned
// around: in global memory a lane has 16 bytes of a token, eight channels; in
// the pass it has a channel and all tokens.  Element pairs go through
// ldmatrix / stmatrix with transposition: matrix m of eight tokens takes
// channels 8 j + 2 m, + 1 from the lanes with lane % 4 = j, so that a lane's
// four registers are its 16 bytes.  A channel's row is 64 bytes in 16-byte
// units; unit i is at i ^ turn_swap(channel), which puts the eight rows of a
// matrix, and eight neighbouring channels, into different banks.
__device__ __forceinline__ int turn_swap(int ch) { return ((ch >> 1) ^ (ch >> 3)) & 3; }
struct Turn {
    uint8_t* mine;          // this lane's channel's row
    uint32_t matrix;        // shared address of the row that this lane names for ldmatrix / stmatrix
    int mine_swap, matrix_swap;
    int token, channel;     // of this lane's 16 bytes: token of eight, first channel
};
__device__ __forceinline__ Turn turn_of(uint8_t* area) {
    const int warp = (threadIdx.x >> 5) & 7, lane = threadIdx.x & 31, m = lane >> 3, r = lane & 7;
    const int ch = 8 * (r >> 1) + 2 * m + (r & 1);
    uint8_t* tile = area + warp * 2048;
    Turn t;
    t.mine = tile + lane * 64;
    t.mine_swap = turn_swap(lane);
    t.matrix = umma::smem_u32(tile + ch * 64);
    t.matrix_swap = turn_swap(ch);
    t.token = (warp >> 2) * kHalf + (lane >> 2);
    t.channel = (warp & 3) * 32 + (lane & 3) * 8;
    return t;
}
__device__ __forceinline__ void load_tokens(const TcArgs& a, const Episode& w, const Turn& t, int c, uint4 (&v)[4]) {
    const bool in = c >= 0 && t.channel < a.shape.v_dim;
    const __nv_bfloat16* from = a.rows + ((int64_t)w.sp.start + (int64_t)c * kChunk + t.token) * a.row_stride +
                                (int64_t)w.head * a.shape.v_dim + t.channel;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = make_uint4(0, 0, 0, 0);
        if (in && c * kChunk + t.token + 8 * i < w.sp.len)
            v[i] = __ldg(reinterpret_cast<const uint4*>(from + (int64_t)(8 * i) * a.row_stride));
    }
}
__device__ __forceinline__ void turn_in(const Turn& t, const uint4 (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                         t.matrix + ((i ^ t.matrix_swap) << 4)),
                     "r"(v[i].x), "r"(v[i].y), "r"(v[i].z), "r"(v[i].w)
                     : "memory");
    __syncwarp();
}
// Tokens 8 i .. 8 i + 7 of this lane's channel.
__device__ __forceinline__ void eight_tokens(const Turn& t, int i, float (&x)[8]) {
    const uint4 q = *reinterpret_cast<const uint4*>(t.mine + ((i ^ t.mine_swap) << 4));
    const uint32_t r[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int z = 0; z < 4; ++z) {
        x[2 * z] = __uint_as_float(r[z] << 16);
        x[2 * z + 1] = __uint_as_float(r[z] & 0xffff0000u);
    }
}
// h: this channel's tokens in pairs.
__device__ __forceinline__ void store_tokens(const TcArgs& a, const Episode& w, const Turn& t, int c,
                                             const uint32_t (&h)[kHalf / 2]) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4*>(t.mine + ((i ^ t.mine_swap) << 4)) =
            make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
    __syncwarp();
    const bool in = t.channel < a.shape.v_dim;
    __nv_bfloat16* to = a.out + ((int64_t)w.sp.start + (int64_t)c * kChunk + t.token) * a.out_stride +
                        (int64_t)w.head * a.shape.v_dim + t.channel;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint4 q;
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                     : "r"(t.matrix + ((i ^ t.matrix_swap) << 4))
                     : "memory");
        if (in && c * kChunk + t.token + 8 * i < w.sp.len)
            *reinterpret_cast<uint4*>(to + (int64_t)(8 * i) * a.out_stride) = q;
    }
    __syncwarp();
}

// Values of a vector at N columns.
template <int N>
__device__ __forceinline__ void cols_of(const float* vec, int which, int c, float (&x)[N]) {
#pragma unroll
    for (int z = 0; z < N; z += 4) {
        const float4 v = *reinterpret_cast<const float4*>(vec + which * kChunk + c + z);
        x[z] = v.x;
        x[z + 1] = v.y;
        x[z + 2] = v.z;
        x[z + 3] = v.w;
    }
}

// N columns of a row of a state, from column `col`.
template <int N>
__device__ __forceinline__ void load_row(const float* from, float (&s)[N], int row, int col, int dv, int dk) {
#pragma unroll
    for (int c = 0; c < N; c += 4) {
        float4 v = make_float4(0, 0, 0, 0);
        if (from != nullptr && row < dv && col + c < dk)
            v = *reinterpret_cast<const float4*>(from + (int64_t)row * dk + col + c);
        s[c] = v.x;
        s[c + 1] = v.y;
        s[c + 2] = v.z;
        s[c + 3] = v.w;
    }
}

__device__ __forceinline__ void init_bars(Bars& b) {
    if (threadIdx.x == 0) {
        uint64_t* all[] = {&b.full[0], &b.full[1], &b.s_ready, &b.u_ready, &b.free, &b.a,
                           &b.b,       &b.t,       &b.s,       &b.p,       &b.done[0], &b.done[1]};
        for (uint64_t* m : all) umma::mbar_init(m, 1);
        b.dead = 0;
        b.copied = 0;
        umma::fence_mbar_init();
    }
}

// End of a CTA.  After a wait that gave up, products and copies may still be on
// their way: they are waited for, again with a limit, before TMEM and shared
// memory are given back.
__device__ __forceinline__ void finish(const TcArgs& a, Bars& b, uint32_t tmem) {      // all warps have met
    umma::fence_after_sync();
    if (b.dead) {
        if (threadIdx.x % kTokThreads == 0) {      // the threads that issue the products
            uint64_t* bar = &b.done[threadIdx.x / kTokThreads];
            umma::commit(bar);
            umma::mbar_wait(bar, 0, kWaitNs);
        }
        if (threadIdx.x == 0) {
            for (int n = max(b.copied - 2, 0); n < b.copied; ++n)
                umma::mbar_wait(&b.full[n & 1], (uint32_t)(n >> 1) & 1u, kWaitNs);
            atomicAdd(a.status + OFRL_STAT_TIMEOUT, 1);
        }
        __syncthreads();
    }
    if (threadIdx.x < 32) umma::tmem_dealloc(tmem, 512);
}

// The forward pass once more (see delta_redo.cuh), over shared memory and
// images that nothing uses any more.
template <int DK, bool SAVE>
__device__ __forceinline__ void redo_pass(const TcArgs& a, uint8_t* smem) {
    using S = Smem<DK>;
    static_assert(S::kBytes >= redo_bytes<DK>(kRows), "shared memory");
    asm volatile("cp.async.bulk.wait_group 0;\n\tfence.proxy.async;" ::: "memory");      // images on their way
    __syncthreads();
    const Episode w = episode(a, fresh_block());
    const int64_t at = w.slot0 * a.shape.v_heads + w.head;
    Redo r;
    r.tid = (int)fresh_thread();
    r.threads = kThreads;
    r.in = &a.in;
    r.v = a.rows;
    r.v_stride = a.row_stride;
    r.out = a.out;
    r.out_stride = a.out_stride;
    r.sp = w.sp;
    r.skip = 0;
    r.head = w.head;
    r.khead = w.khead;
    r.v_heads = a.shape.v_heads;
    r.dk = a.shape.k_dim;
    r.dv = a.shape.v_dim;
    r.row0 = 0;
    r.rows = kRows;
    r.first = a.first ? a.first + w.states : nullptr;
    r.last = nullptr;
    r.state_img = SAVE ? a.state_img + at * S::kState : nullptr;
    r.vec_img = SAVE ? a.vec_img + at * kTok : nullptr;
    r.state_unit = SAVE ? a.state_unit + at : nullptr;
    r.vec_unit = SAVE ? a.vec_unit + at : nullptr;
    r.pairs = a.pairs + at * kPairBytes;
    r.planes = 1;
    redo_rows<__nv_bfloat16, DK>(r, reinterpret_cast<float*>(smem));
}

// TMEM columns.
constexpr int t_x = 0, t_q = 64, t_u = 128, t_o = 192, t_s = 256, t_s2 = 384;

template <int DK, bool SAVE>
__global__ void __launch_bounds__(kThreads) delta_forward_tc_kernel(const __grid_constant__ TcArgs a) {
    using S = Smem<DK>;
    constexpr int CG = DK / 8, KS = DK / 16, NS = DK / 2;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(16) Bars b;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = threadIdx.x & 127, half = (warp >> 2) & 1;
    const Episode w = episode(a, blockIdx.x);
    const int dk = a.shape.k_dim, dv = a.shape.v_dim;
    init_bars(b);
    // before the wait below: the kernel before lets this one go when all its CTAs have their TMEM
    if (warp == 0) umma::tmem_alloc(&b.tmem, 512);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = b.tmem, mine = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t base = umma::smem_u32(smem);
    const int at_row = (row >> 3) * kTile + (row & 7) * 16;      // of a row in an operand image
    const int col = half * kHalf, at = at_row + half * (kHalf / 8) * kCol;      // of its tokens
    float* row_most = reinterpret_cast<float*>(smem + S::off_row);
    auto vec_of = [&](int n) {
        return reinterpret_cast<const float*>(smem + S::off_stage + (n & 1) * S::kStage + 2 * S::kKey + 2 * kSquare);
    };
    auto keys_at = [&](int n) { return base + S::off_stage + (n & 1) * S::kStage; };

    bool finite = true;
    if (threadIdx.x < kTokThreads) {
        const Turn turn = turn_of(smem + S::off_turn);
        uint4 v[4];
        load_tokens(a, w, turn, 0, v);
        constexpr uint32_t kIdT = umma::instr_desc(umma::kTypeF16, false, true, kRows, kChunk);
        constexpr uint32_t kIdP = umma::instr_desc(umma::kTypeF16, false, false, kRows, kChunk);
        constexpr uint32_t kIdS = umma::instr_desc(umma::kTypeF16, false, true, kRows, DK);
        pdl_wait();
        for (int n = 0; n < w.chunks; ++n) {
            const float* vec = vec_of(n);
            const uint32_t pair = keys_at(n) + 2 * S::kKey;
            turn_in(turn, v);
            wait(b, &b.full[n & 1], n >> 1);
            float x[kHalf];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float f[8], t[8];
                cols_of(vec, V_XV, col + 8 * i, f);
                eight_tokens(turn, i, t);
#pragma unroll
                for (int z = 0; z < 8; ++z) x[8 * i + z] = f[z] * t[z];
            }
            wait(b, &b.s_ready, n);
            wait(b, &b.a, n);
            const float s_inv = b.s_inv;
            {
                float y[kHalf];
                tmem_row(mine + t_x + col, y);
#pragma unroll
                for (int c = 0; c < kHalf; c += 4) {
                    float g[4];
                    cols_of(vec, V_XS, col + c, g);
#pragma unroll
                    for (int z = 0; z < 4; ++z) x[c + z] -= (g[z] * s_inv) * y[c + z];
                }
            }
            row_most[half * kRows + row] = half_max(x);
            group_sync<1>();
            const float x_up = scale_up(fmaxf(row_most[row], row_most[kRows + row])), x_inv = pow2_inv(x_up);
            put_cols(smem + S::off_a + at, x, x_up);
            umma::fence_smem_to_async();
            umma::fence_before_sync();
            group_sync<1>();
            umma::fence_after_sync();
            if (threadIdx.x == 0) {
                mma_run(tmem + t_u, umma::smem_desc(base + S::off_a, kCol, kTile), 2 * kCol,
                        umma::smem_desc(pair, 8 * kTile, kTile), 2 * 8 * kTile, kIdT, 4);
                umma::commit(&b.t);
                if (SAVE) umma::bulk_wait_read();      // U's image of the chunk before
            }
            __syncwarp();
            wait(b, &b.t, n);
            tmem_row(mine + t_u + col, x);
            const float u_max = group_max_nan<1>(b.most[0], half_max_nan(x) * x_inv), u_up = scale_up(u_max);
            finite &= u_max < INFINITY;
            const float u_inv = pow2_inv(u_up), u_f = u_up * x_inv;
            {
                // rest U, with a power of two of its own where states grow
                const float r_up = scale_up(u_max * vec[V_MISC * kChunk + kMost]), r_f = r_up * x_inv;
                if (threadIdx.x == 0) b.r_inv = pow2_inv(r_up);
                float y[kHalf];
#pragma unroll
                for (int c = 0; c < kHalf; c += 4) {
                    float f[4];
                    cols_of(vec, V_REST, col + c, f);
#pragma unroll
                    for (int z = 0; z < 4; ++z) y[c + z] = x[c + z] * f[z];
                }
                put_cols(smem + S::off_c + at, y, r_f);
            }
            if (threadIdx.x == 0) b.u_inv = u_inv;
            umma::fence_smem_to_async();
            umma::fence_before_sync();
            group_sync<1>();
            umma::fence_after_sync();
            if (threadIdx.x == 0) {
                umma::mbar_arrive(&b.u_ready);
                mma_run(tmem + t_s, umma::smem_desc(base + S::off_c, kCol, kTile), 2 * kCol,
                        umma::smem_desc(keys_at(n), CG * kTile, kTile), 2 * CG * kTile, kIdS, 4);
                umma::commit(&b.s);
            }
            __syncwarp();
            load_tokens(a, w, turn, n + 1, v);
            if (n > 0) wait(b, &b.p, n - 1);      // what read the image below is done
            put_cols(smem + S::off_b + at, x, u_f);
            umma::fence_smem_to_async();
            umma::fence_before_sync();
            group_sync<1>();
            umma::fence_after_sync();
            if (warp == 0) {
                wait(b, &b.free, n);
                if (lane == 0) {
                    mma_run(tmem + t_o, umma::smem_desc(base + S::off_b, kCol, kTile), 2 * kCol,
                            umma::smem_desc(pair + kSquare, kTile, 8 * kTile), 2 * kTile, kIdP, 4);
                    umma::commit(&b.p);
                    if (SAVE) {
                        const int64_t to = (w.slot0 + n) * a.shape.v_heads + w.head;
                        umma::bulk_s2g(a.vec_img + to * kTok, smem + S::off_b, kTok);
                        umma::bulk_commit();
                        a.vec_unit[to] = u_inv;
                    }
                }
                __syncwarp();
            }
        }
        if (SAVE && threadIdx.x == 0) umma::bulk_wait_read();
    } else {
        // Turn n: the state before chunk n; then the outputs of chunk n - 1.
        const Turn turn = turn_of(smem + S::off_d);
        float s[NS], inv = 0.0f, u_inv = 0.0f;
        const int s_col = half * NS;
        uint8_t* mine_s = smem + S::off_s + at_row + half * (NS / 8) * kCol;
        load_row(a.first ? a.first + w.states : nullptr, s, row, s_col, dv, dk);
        pdl_wait();
        if (threadIdx.x == kTokThreads && w.chunks > 0) copy_stage<DK>(a, w, smem, b, 0, 0);
        constexpr uint32_t kIdA = umma::instr_desc(umma::kTypeF16, false, false, kRows, kChunk);
        for (int n = 0; n <= w.chunks && w.chunks > 0; ++n) {
            const float inv_before = inv;
            if (n > 0) {
                wait(b, &b.full[(n - 1) & 1], (n - 1) >> 1);
                wait(b, &b.u_ready, n - 1);
                wait(b, &b.s, n - 1);
                u_inv = b.u_inv;
            }
            if (n < w.chunks) {
                if (n > 0) {
                    const float keep = vec_of(n - 1)[V_GAM * kChunk + kChunk - 1], r_inv = b.r_inv;
#pragma unroll
                    for (int c = 0; c < NS; c += 32) {
                        float d[32];
                        tmem_row(mine + t_s + s_col + c, d);
#pragma unroll
                        for (int z = 0; z < 32; ++z) s[c + z] = keep * s[c + z] + r_inv * d[z];
                    }
                    wait(b, &b.b, n - 1);      // what read the image is done
                }
                if (SAVE && threadIdx.x == kTokThreads) umma::bulk_wait_read();      // the image of the chunk before
                const float up = scale_up(group_max<2>(b.most[1], half_max(s)));
                inv = pow2_inv(up);
                put_cols(mine_s, s, up);
                if (threadIdx.x == kTokThreads) b.s_inv = inv;
                umma::fence_smem_to_async();
                umma::fence_before_sync();
                group_sync<2>();
                umma::fence_after_sync();
                if (warp == kTokThreads / 32) {
                    wait(b, &b.full[n & 1], n >> 1);
                    if (lane == 0) {
                        umma::mbar_arrive(&b.s_ready);
                        mma_run(tmem + t_x, umma::smem_desc(base + S::off_s, kCol, kTile), 2 * kCol,
                                umma::smem_desc(keys_at(n), kTile, CG * kTile), 2 * kTile, kIdA, KS);
                        umma::commit(&b.a);
                        if (SAVE) {
                            const int64_t to = (w.slot0 + n) * a.shape.v_heads + w.head;
                            umma::bulk_s2g(a.state_img + to * S::kState, smem + S::off_s, S::kState);
                            umma::bulk_commit();
                            a.state_unit[to] = inv;
                        }
                    }
                    __syncwarp();
                }
            }
            if (n > 0) {
                const float* vec = vec_of(n - 1);
                wait(b, &b.b, n - 1);
                wait(b, &b.p, n - 1);
                const float p_inv = u_inv * vec[V_MISC * kChunk + kPUnit];
                uint32_t h[kHalf / 2];
#pragma unroll
                for (int c = 0; c < kHalf; c += 16) {
                    float x[16], o[16], f[16], g[16];
                    umma::tmem_ld16(mine + t_q + col + c, x);
                    umma::tmem_ld16(mine + t_o + col + c, o);
                    umma::tmem_ld_wait();
                    cols_of(vec, V_OS, col + c, f);
                    cols_of(vec, V_QS, col + c, g);
#pragma unroll
                    for (int z = 0; z < 16; ++z) o[z] = (f[z] * inv_before) * x[z] + (g[z] * p_inv) * o[z];
#pragma unroll
                    for (int z = 0; z < 16; z += 2) h[(c + z) / 2] = pack_b(o[z], o[z + 1]);
                }
                store_tokens(a, w, turn, n - 1, h);
            }
            umma::fence_before_sync();
            group_sync<2>();
            umma::fence_after_sync();
            if (threadIdx.x == kTokThreads && n < w.chunks) {
                umma::mbar_arrive(&b.free);
                mma_run(tmem + t_q, umma::smem_desc(base + S::off_s, kCol, kTile), 2 * kCol,
                        umma::smem_desc(keys_at(n) + S::kKey, kTile, CG * kTile), 2 * kTile, kIdA, KS);
                umma::commit(&b.b);
                if (n + 1 < w.chunks) copy_stage<DK>(a, w, smem, b, n + 1, n + 1);
            }
            __syncwarp();
        }
        if (SAVE && threadIdx.x == kTokThreads) umma::bulk_wait_read();
    }
    if (__syncthreads_or(!finite) && !b.dead) redo_pass<DK, SAVE>(a, smem);
    finish(a, b, tmem);
}

template <int DK>
__global__ void __launch_bounds__(kThreads) delta_reverse_tc_kernel(const __grid_constant__ TcArgs a) {
    using S = Smem<DK>;
    constexpr int CG = DK / 8, KS = DK / 16, NS = DK / 2;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(16) Bars b;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = threadIdx.x & 127, half = (warp >> 2) & 1;
    pdl_wait();
    pdl_trigger();
    const Episode w = episode(a, blockIdx.x);
    const int dk = a.shape.k_dim, dv = a.shape.v_dim;
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.counter = 0;
    init_bars(b);
    if (warp == 0) umma::tmem_alloc(&b.tmem, 512);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = b.tmem, mine = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t base = umma::smem_u32(smem);
    const int at_row = (row >> 3) * kTile + (row & 7) * 16;      // of a row in an operand image
    const int col = half * kHalf, at = at_row + half * (kHalf / 8) * kCol;      // of its tokens
    float* row_most = reinterpret_cast<float*>(smem + S::off_row);
    auto vec_of = [&](int n) {
        return reinterpret_cast<const float*>(smem + S::off_stage + (n & 1) * S::kStage + 2 * S::kKey + 2 * kSquare);
    };
    auto keys_at = [&](int n) { return base + S::off_stage + (n & 1) * S::kStage; };

    if (threadIdx.x < kTokThreads) {
        // dO is turned around in the place of its operand
        const Turn turn = turn_of(smem + S::off_a);
        uint4 v[4];
        load_tokens(a, w, turn, w.chunks - 1, v);
        constexpr uint32_t kIdP = umma::instr_desc(umma::kTypeF16, false, true, kRows, kChunk);
        constexpr uint32_t kIdT = umma::instr_desc(umma::kTypeF16, false, false, kRows, kChunk);
        constexpr uint32_t kIdS = umma::instr_desc(umma::kTypeF16, false, true, kRows, DK);
        for (int n = 0; n < w.chunks; ++n) {
            const int c0 = w.chunks - 1 - n;
            const float* vec = vec_of(n);
            const uint32_t pair = keys_at(n) + 2 * S::kKey;
            float* u_most = row_most + (n & 1) * 2 * kRows;
            turn_in(turn, v);
            wait(b, &b.full[n & 1], n >> 1);
            // dO scale kq, for P; and times gamma, for the state
            float x[kHalf], y[kHalf];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float f[8], g[8], t[8];
                cols_of(vec, V_QS, col + 8 * i, f);
                cols_of(vec, V_GAM, col + 8 * i, g);
                eight_tokens(turn, i, t);
#pragma unroll
                for (int z = 0; z < 8; ++z) {
                    x[8 * i + z] = t[z] * f[z];
                    y[8 * i + z] = x[8 * i + z] * g[z];
                }
            }
            const float o_most = warp_max(half_max(y));
            if (lane == 0) b.more[warp] = o_most;
            if (threadIdx.x == 0) umma::bulk_wait_read();      // R's image of the chunk before
            const float a_up = scale_up(group_max<1>(b.most[0], half_max(x))), p_inv = pow2_inv(a_up) * vec[V_MISC * kChunk + kPUnit];
            const float o_up = scale_up(all_max(b.more));
            put_cols(smem + S::off_a + at, x, a_up);
            umma::fence_smem_to_async();
            umma::fence_before_sync();
            group_sync<1>();
            umma::fence_after_sync();
            if (threadIdx.x == 0) {
                mma_run(tmem + t_q, umma::smem_desc(base + S::off_a, kCol, kTile), 2 * kCol,
                        umma::smem_desc(pair + kSquare, 8 * kTile, kTile), 2 * 8 * kTile, kIdP, 4);
                umma::commit(&b.b);
                b.o_inv[n & 1] = pow2_inv(o_up);
            }
            __syncwarp();
            if (n > 0) wait(b, &b.s, n - 1);      // what read the image below is done
            put_cols(smem + S::off_c + at, y, o_up);
            wait(b, &b.b, n);
            tmem_row(mine + t_q + col, y);
            wait(b, &b.s_ready, n);
            wait(b, &b.a, n);
            const float s_inv = b.s_inv;
            tmem_row(mine + t_x + col, x);
#pragma unroll
            for (int c = 0; c < kHalf; c += 4) {
                float f[4];
                cols_of(vec, V_REST, col + c, f);
#pragma unroll
                for (int z = 0; z < 4; ++z) x[c + z] = (f[z] * s_inv) * x[c + z] + p_inv * y[c + z];
            }
            u_most[half * kRows + row] = half_max(x);
            group_sync<1>();
            const float u_up = scale_up(fmaxf(u_most[row], u_most[kRows + row])), u_inv = pow2_inv(u_up);
            put_cols(smem + S::off_b + at, x, u_up);
            umma::fence_smem_to_async();
            umma::fence_before_sync();
            group_sync<1>();
            umma::fence_after_sync();
            const uint32_t t_r = (n & 1) ? t_o : t_u;
            if (threadIdx.x == 0) {
                mma_run(tmem + t_r, umma::smem_desc(base + S::off_b, kCol, kTile), 2 * kCol, umma::smem_desc(pair, kTile, 8 * kTile),
                        2 * kTile, kIdT, 4);
                umma::commit(&b.t);
                // beside it: dO's part of the state's next gradient
                mma_run(tmem + t_s, umma::smem_desc(base + S::off_c, kCol, kTile), 2 * kCol,
                        umma::smem_desc(keys_at(n) + S::kKey, CG * kTile, kTile), 2 * CG * kTile, kIdS, 4);
            }
            __syncwarp();
            load_tokens(a, w, turn, c0 - 1, v);
            wait(b, &b.t, n);
            tmem_row(mine + t_r + col, x);
#pragma unroll
            for (int c = 0; c < kHalf; c += 4) {
                float f[4], g[4];
                cols_of(vec, V_TINV, col + c, f);
                cols_of(vec, V_DS, col + c, g);
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    x[c + z] *= f[z] * u_inv;
                    y[c + z] = -x[c + z] * g[z];
                }
            }
            const float i_most = warp_max(half_max(x));
            if (lane == 0) b.more[warp] = i_most;
            const float r_up = scale_up(group_max<1>(b.most[0], half_max(y)));
            const float i_up = scale_up(all_max(b.more));
            if (threadIdx.x == 0) b.r_inv = pow2_inv(r_up);
            put_cols(smem + S::off_d + at, y, r_up);
            umma::fence_smem_to_async();
            umma::fence_before_sync();
            group_sync<1>();
            umma::fence_after_sync();
            if (threadIdx.x == 0) {
                umma::mbar_arrive(&b.u_ready);
                mma_run(tmem + t_s2, umma::smem_desc(base + S::off_d, kCol, kTile), 2 * kCol,
                        umma::smem_desc(keys_at(n), CG * kTile, kTile), 2 * CG * kTile, kIdS, 4);
                umma::commit(&b.s);
            }
            __syncwarp();
            put_cols(smem + S::off_b + at, x, i_up);
            umma::fence_smem_to_async();
            group_sync<1>();
            if (threadIdx.x == 0) {
                const int64_t to = (w.slot0 + c0) * a.shape.v_heads + w.head;
                umma::bulk_s2g(a.vec_img + to * kTok, smem + S::off_b, kTok);
                umma::bulk_commit();
                a.vec_unit[to] = pow2_inv(i_up);
            }
            __syncwarp();
        }
        if (threadIdx.x == 0) umma::bulk_wait_read();
    } else {
        // Turn n (chunks are counted from the last): the state's gradient after
        // chunk n; then dv of chunk n - 1, from the product that the tokens'
        // warps made R of.
        const Turn turn = turn_of(smem + S::off_turn);
        float s[NS];
        const int s_col = half * NS;
        uint8_t* mine_s = smem + S::off_s + at_row + half * (NS / 8) * kCol;
        if (threadIdx.x == kTokThreads && w.chunks > 0) copy_stage<DK>(a, w, smem, b, 0, w.chunks - 1);
        load_row(a.first ? a.first + w.states : nullptr, s, row, s_col, dv, dk);
        constexpr uint32_t kIdA = umma::instr_desc(umma::kTypeF16, false, false, kRows, kChunk);
        for (int n = 0; n <= w.chunks && w.chunks > 0; ++n) {
            const int c0 = w.chunks - 1 - n;
            float* dv_f = b.dv_f[n & 1];
            if (n > 0) {
                const float* vec = vec_of(n - 1);
                wait(b, &b.full[(n - 1) & 1], (n - 1) >> 1);
                const float keep = vec[V_GAM * kChunk + kChunk - 1];
                const int i = threadIdx.x - kTokThreads;
                if (i < kChunk) dv_f[i] = vec[V_TINV * kChunk + i] * vec[V_DV * kChunk + i];
                wait(b, &b.u_ready, n - 1);
                wait(b, &b.s, n - 1);
                const float o_inv = b.o_inv[(n - 1) & 1], r_inv = b.r_inv;
#pragma unroll
                for (int c = 0; c < NS; c += 16) {
                    float d[16], e[16];
                    umma::tmem_ld16(mine + t_s + s_col + c, d);
                    umma::tmem_ld16(mine + t_s2 + s_col + c, e);
                    umma::tmem_ld_wait();
#pragma unroll
                    for (int z = 0; z < 16; ++z) s[c + z] = keep * s[c + z] + (o_inv * d[z] + r_inv * e[z]);
                }
            }
            if (threadIdx.x == kTokThreads) umma::bulk_wait_read();      // the image of the chunk before
            const float up = scale_up(group_max<2>(b.most[1], half_max(s))), inv = pow2_inv(up);
            if (n < w.chunks) {
                // nothing reads the stage of the chunk before any more
                if (threadIdx.x == kTokThreads + 32 && n + 1 < w.chunks) copy_stage<DK>(a, w, smem, b, n + 1, c0 - 1);
                __syncwarp();
                put_cols(mine_s, s, up);
                if (threadIdx.x == kTokThreads) b.s_inv = inv;
                umma::fence_smem_to_async();
                umma::fence_before_sync();
                group_sync<2>();
                umma::fence_after_sync();
                if (warp == kTokThreads / 32) {
                    wait(b, &b.full[n & 1], n >> 1);
                    if (lane == 0) {
                        umma::mbar_arrive(&b.s_ready);
                        mma_run(tmem + t_x, umma::smem_desc(base + S::off_s, kCol, kTile), 2 * kCol,
                                umma::smem_desc(keys_at(n), kTile, CG * kTile), 2 * kTile, kIdA, KS);
                        umma::commit(&b.a);
                        const int64_t to = (w.slot0 + c0) * a.shape.v_heads + w.head;
                        umma::bulk_s2g(a.state_img + to * S::kState, smem + S::off_s, S::kState);
                        umma::bulk_commit();
                        a.state_unit[to] = inv;
                    }
                    __syncwarp();
                }
            }
            if (n > 0) {
                const float* u_most = row_most + ((n - 1) & 1) * 2 * kRows;
                const float u_inv = pow2_inv(scale_up(fmaxf(u_most[row], u_most[kRows + row])));
                const uint32_t t_r = ((n - 1) & 1) ? t_o : t_u;
                uint32_t h[kHalf / 2];
#pragma unroll
                for (int c = 0; c < kHalf; c += 16) {
                    float x[16], f[16];
                    umma::tmem_ld16(mine + t_r + col + c, x);
                    umma::tmem_ld_wait();
#pragma unroll
                    for (int z = 0; z < 16; z += 4) {
                        const float4 q = *reinterpret_cast<const float4*>(dv_f + col + c + z);
                        f[z] = q.x, f[z + 1] = q.y, f[z + 2] = q.z, f[z + 3] = q.w;
                    }
#pragma unroll
                    for (int z = 0; z < 16; z += 2) h[(c + z) / 2] = pack_b(x[z] * (f[z] * u_inv), x[z + 1] * (f[z + 1] * u_inv));
                }
                umma::fence_before_sync();
                store_tokens(a, w, turn, c0 + 1, h);
            }
        }
        if (threadIdx.x == kTokThreads) umma::bulk_wait_read();
        if (a.last && row < dv) {
            float* to = a.last + w.states + (int64_t)row * dk;
#pragma unroll
            for (int c = 0; c < NS; c += 4)
                if (s_col + c < dk) *reinterpret_cast<float4*>(to + s_col + c) = make_float4(s[c], s[c + 1], s[c + 2], s[c + 3]);
        }
    }
    __syncthreads();
    finish(a, b, tmem);
}

template <auto KERNEL, int DK>
cudaError_t go(const TcArgs& c, int64_t grid, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    const cudaError_t e = opt_in(KERNEL, Smem<DK>::kBytes, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(KERNEL, dim3((unsigned)grid), dim3(kThreads), Smem<DK>::kBytes, st, c);
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
        return a.saved ? go<delta_forward_tc_kernel<128, true>, 128>(c, grid, st)
                       : go<delta_forward_tc_kernel<128, false>, 128>(c, grid, st);
    return a.saved ? go<delta_forward_tc_kernel<64, true>, 64>(c, grid, st)
                   : go<delta_forward_tc_kernel<64, false>, 64>(c, grid, st);
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
    return a.shape.k_dim > 64 ? go<delta_reverse_tc_kernel<128>, 128>(c, grid, st)
                              : go<delta_reverse_tc_kernel<64>, 64>(c, grid, st);
}

}  // namespace delta
}  // namespace ofrl
