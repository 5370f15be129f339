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
// nothing but a largest magnitude passes between warps.  Bulk copies keep a
// ring of stages filled.  (A fifth warp for the copies lost: it leaves three
// warps on one register file, 168 registers each.)
//
// Bound by the latency of a chunk's products and conversions, one after the
// other: 3 us a chunk of 64 x 64 with one plane, 64 episodes of 256 tokens and
// two heads 11.5 us forward, 13 when it saves, and 13.5 us back (24 and 23 us
// with two planes).  Leaving out the zero blocks of T and P took 3 to 10% off.

#include <algorithm>
#include <cmath>

#include "delta_redo.cuh"

namespace ofrl {
namespace delta {
namespace {

// NW: computing warps of a CTA, 16 value channels each.
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
    float* state_unit;       // [slot][head]: their powers of two
    float* vec_unit;
    int32_t stages;          // of the ring
    // forward over parts of an episode (segments > 1)
    int32_t segments;
    float* seg_state;        // [episode][head][segments][v_dim][k_dim] states at the parts' starts
    uint8_t* seg_map;        // [episode][head][segments] images of the parts' maps, two planes
    float* seg_unit;         // [episode][head][segments][8] their powers of two per 16 rows
    unsigned* counter;       // backward: zeroed for the gradient kernel
    int32_t* status;
};

// One stage of the ring: K^ and Q^ planes, T^T / P / vectors (/ second planes).
// Beside the ring each warp has two buffers of its token rows (64 tokens, 16
// channels) and, for bf16, one to turn its outputs around.
template <typename T, int DK, int NM, int NW>
struct Stage {
    static constexpr int NT = sizeof(T) == 4 ? 2 : 1;
    static constexpr int kKey = kChunk * DK * 2;
    static constexpr int kKeys = 2 * NT * kKey;
    static constexpr int kPairs = NM == 2 ? (int)kPairBytes : (int)kPairFirst;
    static constexpr int kBytes = kKeys + kPairs;
    static constexpr int kPitch = 16 * (int)sizeof(T) + 16;      // of a token's channels: no bank conflicts
    static constexpr int kRows = kChunk * kPitch;
    static constexpr int kWarp = (sizeof(T) == 2 ? 3 : 2) * kRows;
    // three stages where two CTAs then share an SM, else two where they fit
    static constexpr int kCount = 3 * kBytes + NW * kWarp <= 111 * 1024   ? 3
                                  : 2 * kBytes + NW * kWarp <= 226 * 1024 ? 2
                                                                          : 1;
    static constexpr int kShared = kCount * kBytes + NW * kWarp;
    static_assert(kShared <= 226 * 1024, "shared memory");
    // what goes over an episode again takes its place
    static_assert(kBytes + NW * kWarp >= redo_bytes<DK>(NW * 16), "shared memory");
};

// Token rows of one chunk, transposed: x[t][z] = row value at (channel row4 +
// (z >> 1) * 8 of the warp, token 8 t + col2 + (z & 1)).
template <typename T, int PITCH>
__device__ __forceinline__ void load_transposed(const uint8_t* rows, float (&x)[8][4]) {
    const int lane = threadIdx.x & 31;
    if constexpr (sizeof(T) == 2) {
        const int m = lane >> 3, r = lane & 7;
#pragma unroll
        for (int t = 0; t < 8; t += 2) {
            uint32_t f[4];   // matrices: (token group t + (m >> 1), channel half m & 1)
            ldsm4t(f, umma::smem_u32(rows) + ((t + (m >> 1)) * 8 + r) * PITCH + (m & 1) * 16);
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
                x[t][z] = *reinterpret_cast<const float*>(rows + (t * 8 + col2 + (z & 1)) * PITCH +
                                                          (row4 + (z >> 1) * 8) * 4);
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
    int e, head, khead, row0;      // row0: the CTA's first value channel
    int seg;
    Span sp;                       // of the CTA's part of the episode
    int chunks;
    int64_t slot0;
};
// A CTA's rows, part, head and episode, rows changing fastest.
__device__ __forceinline__ Work work_of(const ChainArgs& a, unsigned block, int slices, int width, int segments, int in_all) {
    Work w;
    const int hv = a.shape.v_heads;
    w.row0 = block % slices * width;
    w.seg = block / slices % segments;
    const int64_t item = block / slices / segments;
    w.e = (int)(item / hv);
    w.head = (int)(item % hv);
    w.khead = w.head / (hv / a.shape.k_heads);
    w.sp = span_of(a.ends, w.e, (int32_t)a.in.tokens);
    w.chunks = (w.sp.len + kChunk - 1) / kChunk;
    w.slot0 = w.sp.start / kChunk + w.e;
    if (in_all > 1) {      // the episode's chunks in equal parts, the last ones perhaps empty
        const int per = (w.chunks + in_all - 1) / in_all, from = min(w.seg * per, w.chunks);
        w.chunks = min(per, w.chunks - from);
        w.sp.start += from * kChunk;
        w.sp.len = min(w.sp.len - from * kChunk, w.chunks * kChunk);
        w.slot0 += from;
    }
    return w;
}

// Barriers of a CTA's ring, and what its computing warps exchange.
struct Ring {
    uint64_t full[3], empty[3];
    int dead;             // a wait gave up
    int copied;           // turns whose copies were started
    float most[2][8];     // per warp: largest magnitudes
};

template <int NW>
__device__ __forceinline__ void ring_init(Ring& r) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < 3; ++i) {
            umma::mbar_init(&r.full[i], 1);
            umma::mbar_init(&r.empty[i], NW);
        }
        r.dead = 0;
        r.copied = 0;
        umma::fence_mbar_init();
    }
    __syncthreads();
}

// The first warp fills the ring: the copies of turn n of the pass, once every
// warp is done with what its stage held.  (A warp for the copies alone would
// leave three warps on one of the SM's four register files, and a third of
// the registers of every warp unused.)
template <typename St, int DK, bool REVERSE>
__device__ __forceinline__ void copy_chunk(const ChainArgs& a, const Work& w, uint8_t* smem, Ring& r, int n, int st,
                                           int before) {
    if (n >= w.chunks) return;
    const int c = REVERSE ? w.chunks - 1 - n : n;
    // lanes may see another warp set `dead` at different times: they decide together
    bool ok = !*(volatile int*)&r.dead;
    if (ok && before >= 0) ok = umma::mbar_wait(&r.empty[st], (uint32_t)before & 1u, kWaitNs);
    if (__any_sync(0xffffffffu, !ok)) {
        r.dead = 1;
        return;
    }
    if ((threadIdx.x & 31) == 0) {
        r.copied = n + 1;
        uint8_t* s = smem + st * St::kBytes;
        const int64_t slot = w.slot0 + c;
        umma::mbar_expect_tx(&r.full[st], (uint32_t)St::kBytes);
        umma::bulk_g2s(s, a.keys + (slot * a.shape.k_heads + w.khead) * KeyImage::bytes(DK, St::NT), St::kKeys, &r.full[st]);
        umma::bulk_g2s(s + St::kKeys, a.pairs + (slot * a.shape.v_heads + w.head) * kPairBytes, St::kPairs, &r.full[st]);
    }
    __syncwarp();
}

// A warp's own token rows of chunk c: asynchronous 16-byte copies, one group
// per chunk whether or not there is anything to copy.
template <typename St, typename T>
__device__ __forceinline__ void copy_rows(const ChainArgs& a, const Work& w, uint8_t* to, int c, int row0) {
    if (c >= 0 && c < w.chunks) {
        const int lane = threadIdx.x & 31;
        const int rows = min(kChunk, w.sp.len - c * kChunk);
        constexpr int kVecs = sizeof(T);      // 16-byte pieces of 16 channels: 2 or 4
        const int piece = lane % kVecs;
        const bool on = row0 + piece * (16 / (int)sizeof(T)) < a.shape.v_dim;
        const T* from = static_cast<const T*>(a.rows) + ((int64_t)w.sp.start + c * kChunk) * a.row_stride +
                        (int64_t)w.head * a.shape.v_dim + row0 + piece * (16 / sizeof(T));
        const uint32_t dst = umma::smem_u32(to) + piece * 16;
#pragma unroll
        for (int i = 0; i < kChunk * kVecs / 32; ++i) {
            const int row = lane / kVecs + i * (32 / kVecs);
            if (on && row < rows)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + row * St::kPitch),
                             "l"(from + row * a.row_stride)
                             : "memory");
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}
__device__ __forceinline__ void rows_ready() {      // all but the newest group
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncwarp();
}

// Wait of a computing warp for a stage.  After a wait that gave up nothing
// waits any more: the pass runs on over what shared memory holds (warps that
// meet at a barrier all get there) and the CTA reports it.
__device__ __forceinline__ void stage_ready(Ring& r, int st, int turn) {
    const bool ok = *(volatile int*)&r.dead || umma::mbar_wait(&r.full[st], (uint32_t)turn & 1u, kWaitNs);
    if (__any_sync(0xffffffffu, !ok)) r.dead = 1;
    __syncwarp();
}

// End of a CTA.  After a wait that gave up, copies may still be on their way
// into its shared memory: those of the ring's last turns are waited for, again
// with a limit, and the token rows' without one.
__device__ __forceinline__ void ring_end(const ChainArgs& a, Ring& r, int stages) {
    __syncthreads();
    if (!r.dead) return;
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (threadIdx.x != 0) return;
    for (int n = max(r.copied - stages, 0); n < r.copied; ++n)
        umma::mbar_wait(&r.full[n % stages], (uint32_t)(n / stages) & 1u, kWaitNs);
    atomicAdd(a.status + OFRL_STAT_TIMEOUT, 1);
}

// Largest of the computing warps' values (which: 0 and 1 in turn).
template <int NW>
__device__ __forceinline__ float across(Ring& r, int which, float v) {
    if ((threadIdx.x & 31) == 0) r.most[which][threadIdx.x >> 5] = v;
    asm volatile("bar.sync 1, %0;" ::"n"(NW * 32) : "memory");
    float m = r.most[which][0];
#pragma unroll
    for (int i = 1; i < NW; ++i) m = fmaxf(m, r.most[which][i]);
    return m;
}

// Zero what was never copied: tokens past the chunk's end, channels past v_dim.
__device__ __forceinline__ void mask_rows(float (&x)[8][4], int rows, int channels) {
    const int lane = threadIdx.x & 31, row4 = lane >> 2, col2 = (lane & 3) * 2;
    if (rows == kChunk && channels >= 16) return;
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int z = 0; z < 4; ++z)
            if (t * 8 + col2 + (z & 1) >= rows || row4 + (z >> 1) * 8 >= channels) x[t][z] = 0.0f;
}

template <int NA, int NB, int KA>
__device__ __forceinline__ void first_planes(const uint32_t (&a)[NA][KA][4], uint32_t (&b)[NB][KA][4]) {
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int k = 0; k < KA; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) b[n][k][i] = a[n][k][i];
}

// s[t] = keep s[t] + inv (f b [+ g h]) for the tiles of a state, four at a time.
template <int DK, int NM, int NT, bool TWO>
__device__ __forceinline__ void update_state(float (&s)[DK / 8][4], float keep, float inv, const uint32_t (&f)[NM][4][4],
                                             uint32_t b, const uint32_t (&g)[NM][4][4], uint32_t h) {
#pragma unroll
    for (int t = 0; t < DK / 8; t += 4) {
        float d[4][4];
        zero(d);
        gemm<4, 4, NM, NT, true>(d, f, b, kChunk * DK * 2, DK / 8, t);
        if constexpr (TWO) gemm<4, 4, NM, NT, true>(d, g, h, kChunk * DK * 2, DK / 8, t);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int z = 0; z < 4; ++z) s[t + i][z] = keep * s[t + i][z] + inv * d[i][z];
    }
}

template <int NW>
constexpr int min_ctas() { return NW == 4 ? 2 : 1; }

// What a forward pass leaves.  kOutputs: outputs, of a whole episode or of a
// part that starts from seg_state.  kSave: also S and U as images for the
// backward pass; the CTA then has every value channel, so that an image has
// one power of two.  kSummary: of a part, no outputs but what it does to any
// state before it, S -> S M + B: the recurrence is linear, so B is its end
// from the zero state and the rows of M are its ends from the unit vectors
// with v = 0.  The value channels and after them the rows of M are the
// pass's rows.  The first part starts from the episode's own state and needs
// no M.
enum Pass { kOutputs, kSave, kSummary };

// The pass once more (see delta_redo.cuh), over shared memory that nothing uses
// any more.  A part of an episode is gone over from the episode's beginning: its
// own start comes from summaries that were not finite either, which also spoils
// what has one power of two with them.  (The first part's start is kept beside the
// others: the caller's buffer may be that of the final states.)
//
// Registers kept for this over the pass are registers that the pass lacks, so
// what it needs is worked out anew.  Reading block and thread anew too lets the
// 64-wide and the one-plane passes keep their registers as they were; the 128-wide
// ones with two planes then spill 220 bytes, 28 without.
template <typename T, int DK, int NM, int NW, int PASS>
__device__ __forceinline__ void redo_pass(const ChainArgs& a, uint8_t* smem) {
    constexpr bool SAVE = PASS == kSave;
    constexpr int NO = sizeof(T) == 4 ? 2 : 1;
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    const int hv = a.shape.v_heads, dk = a.shape.k_dim, dv = a.shape.v_dim;
    constexpr bool kFresh = DK == 64 || NM == 1;
    const Work w = work_of(a, kFresh ? fresh_block() : blockIdx.x, (dv + NW * 16 - 1) / (NW * 16), NW * 16, a.segments, a.segments);
    const int64_t item = (int64_t)w.e * hv + w.head, at = w.slot0 * hv + w.head;
    Redo r;
    r.tid = (int)(kFresh ? fresh_thread() : threadIdx.x);
    r.threads = NW * 32;
    r.in = &a.in;
    r.v = a.rows;
    r.v_stride = a.row_stride;
    r.out = a.out;
    r.out_stride = a.out_stride;
    r.sp = span_of(a.ends, w.e, (int32_t)a.in.tokens);
    r.skip = w.sp.start - r.sp.start;
    r.sp.len = r.skip + w.sp.len;
    r.head = w.head;
    r.khead = w.khead;
    r.v_heads = hv;
    r.dk = dk;
    r.dv = dv;
    r.row0 = w.row0;
    r.rows = NW * 16;
    r.first = a.segments > 1 ? a.seg_state + item * a.segments * dv * dk : a.first ? a.first + item * dv * dk : nullptr;
    r.last = a.last && w.seg == a.segments - 1 ? a.last + item * dv * dk : nullptr;
    r.state_img = SAVE ? a.state_img + at * NO * NW * 16 * DK * 2 : nullptr;
    r.vec_img = SAVE ? a.vec_img + at * NO * NW * 16 * kChunk * 2 : nullptr;
    r.state_unit = SAVE ? a.state_unit + at : nullptr;
    r.vec_unit = SAVE ? a.vec_unit + at : nullptr;
    r.pairs = a.pairs + at * kPairBytes;
    r.planes = NO;
    redo_rows<T, DK>(r, reinterpret_cast<float*>(smem));
}

// NM: planes of S, X, U (and of T and P).
template <typename T, int DK, int NM, int NW, int PASS>
__global__ void __launch_bounds__(NW * 32, min_ctas<NW>()) delta_forward_kernel(const __grid_constant__ ChainArgs a) {
    using St = Stage<T, DK, NM, NW>;
    constexpr int NT = St::NT, CG = DK / 8, KS = DK / 16;
    constexpr int NO = NT;      // planes of the operands that only the outputs see, and of the saved images
    constexpr bool SAVE = PASS == kSave, SUMMARY = PASS == kSummary;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Ring ring;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int v_pad = (a.shape.v_dim + NW * 16 - 1) / (NW * 16) * (NW * 16);
    const Work w = work_of(a, blockIdx.x, (SUMMARY ? v_pad + DK : v_pad) / (NW * 16), NW * 16, SUMMARY ? a.segments - 1 : a.segments,
                           a.segments);
    ring_init<NW>(ring);
    const int stages = a.stages;
    uint8_t* mine = smem + stages * St::kBytes + warp * St::kWarp;
    {
        const int dk = a.shape.k_dim, dv = a.shape.v_dim, hv = a.shape.v_heads;
        const int row0 = w.row0 + warp * 16;
        const int64_t states = ((int64_t)w.e * hv + w.head) * dv * dk;
        float S[DK / 8][4];
        copy_rows<St, T>(a, w, mine, 0, row0);
        const int64_t part = ((int64_t)w.e * hv + w.head) * a.segments + w.seg;
        // the summaries keep a copy of the first part's start: the last part of
        // the pass that follows may write the caller's buffer it came from
        const bool given = SUMMARY ? w.seg == 0 : a.segments == 1;
        if (given) load_state(a.first ? a.first + states : nullptr, S, row0, dv, dk);
        pdl_wait();      // what the launch before leaves
        if (!given) load_state(SUMMARY ? nullptr : a.seg_state + part * dv * dk, S, row0, dv, dk);
        if (SUMMARY && given && row0 < v_pad) store_state(a.seg_state + part * dv * dk, S, row0, dv, dk);
        if (SUMMARY && row0 >= v_pad)
#pragma unroll
            for (int t = 0; t < DK / 8; ++t)
#pragma unroll
                for (int z = 0; z < 4; ++z)
                    S[t][z] = row0 - v_pad + (lane >> 2) + (z >> 1) * 8 == t * 8 + (lane & 3) * 2 + (z & 1) ? 1.0f : 0.0f;
        if (SUMMARY && w.seg == 0 && w.row0 >= v_pad) return;
        if (warp == 0)
            for (int n = 0; n < stages - 1; ++n) copy_chunk<St, DK, false>(a, w, smem, ring, n, n, -1);
        int st = stages - 1, turn = -1;      // of the chunk before
        for (int c = 0; c < w.chunks; ++c) {
            const int st_before = st, turn_before = turn;
            if (++st == stages) st = 0, ++turn;
            copy_rows<St, T>(a, w, mine + ((c + 1) & 1) * St::kRows, c + 1, row0);
            if (stages == 1 && warp == 0) copy_chunk<St, DK, false>(a, w, smem, ring, c, 0, c - 1);
            stage_ready(ring, st, turn);
            if (PASS == kOutputs && row0 >= dv) {
                if (lane == 0) umma::mbar_arrive(&ring.empty[st]);
                continue;
            }
            if (stages > 1 && warp == 0)
                copy_chunk<St, DK, false>(a, w, smem, ring, c + stages - 1, st_before, turn_before);
            const uint8_t* s = smem + st * St::kBytes;
            const uint32_t kimg = umma::smem_u32(s), qimg = kimg + NT * St::kKey, pair = kimg + St::kKeys;
            const float* vec = reinterpret_cast<const float*>(s + St::kKeys + 2 * kSquare);
            const int rows = min(kChunk, w.sp.len - c * kChunk);
            const int64_t at = (w.slot0 + c) * hv + w.head;
            float X[8][4], O[8][4];
            zero(X);
            zero(O);
            float s_max = tile_max(S);
            if constexpr (SAVE) s_max = across<NW>(ring, 0, s_max);
            const float s_up = scale_up(s_max), s_inv = pow2_inv(s_up);
            {
                uint32_t f[NM][KS][4];
                to_frags<NM>(S, s_up, f);
                gemm<KS, 8, NM, NT, false>(X, f, kimg, St::kKey, CG, 0);
                uint32_t f0[NO][KS][4];
                first_planes(f, f0);
                if constexpr (!SUMMARY) gemm<KS, 8, NO, NT, false>(O, f0, qimg, St::kKey, CG, 0);
                if constexpr (SAVE) {
                    const int64_t plane = (int64_t)NW * 16 * DK * 2;
                    store_image<NT == 1 ? 1 : kSliceCols / 8>(a.state_img + at * NO * plane, plane, f0, row0 / 8, NW * 2);
                    if (threadIdx.x == 0) a.state_unit[at] = s_inv;
                }
            }
            {
                float V[8][4];
                rows_ready();
                load_transposed<T, St::kPitch>(mine + (c & 1) * St::kRows, V);
                mask_rows(V, rows, dv - row0);
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    const float2 xv = vec2(vec, V_XV, t), xs = vec2(vec, V_XS, t);
                    const float f[2] = {xv.x, xv.y}, g[2] = {xs.x * s_inv, xs.y * s_inv};
#pragma unroll
                    for (int z = 0; z < 4; ++z) X[t][z] = f[z & 1] * V[t][z] - g[z & 1] * X[t][z];
                }
            }
            float U[8][4];
            zero(U);
            const float x_up = scale_up(tile_max(X)), x_inv = pow2_inv(x_up);
            {
                uint32_t f[NM][4][4];
                to_frags<NM>(X, x_up, f);
                gemm<4, 8, NM, NM, true, kUpper>(U, f, pair, (int)kPairFirst, 8, 0);
            }
            float u_max = tile_max(U) * x_inv;
            if constexpr (SAVE) u_max = across<NW>(ring, 1, u_max);
            const float u_up = scale_up(u_max), u_inv = pow2_inv(u_up), u_f = u_up * x_inv;
            // rest U, with a power of two of its own where states grow
            const float r_up = scale_up(u_max * vec[V_MISC * kChunk + kMost]), r_inv = pow2_inv(r_up), r_f = r_up * x_inv;
            // X now holds rest U, what the state takes in
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const float2 r = vec2(vec, V_REST, t);
                const float f[2] = {r.x * r_f, r.y * r_f};
#pragma unroll
                for (int z = 0; z < 4; ++z) X[t][z] = U[t][z] * f[z & 1];
            }
            if constexpr (!SUMMARY) {
                uint32_t f[NO][4][4];
                to_frags<NO>(U, u_f, f);
                if constexpr (SAVE) {
                    const int64_t plane = (int64_t)NW * 16 * kChunk * 2;
                    store_image<NT == 1 ? 1 : 8>(a.vec_img + at * NO * plane, plane, f, row0 / 8, NW * 2);
                    if (threadIdx.x == 0) a.vec_unit[at] = u_inv;
                }
                zero(U);
                gemm<4, 8, NO, NO, false, kUpper>(U, f, pair + kSquare, (int)kPairFirst, 8, 0);
            }
            if constexpr (!SUMMARY) {
                const float p_inv = u_inv * vec[V_MISC * kChunk + kPUnit];
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    const float2 os = vec2(vec, V_OS, t), qs = vec2(vec, V_QS, t);
                    const float f[2] = {os.x * s_inv, os.y * s_inv}, g[2] = {qs.x * p_inv, qs.y * p_inv};
#pragma unroll
                    for (int z = 0; z < 4; ++z) O[t][z] = f[z & 1] * O[t][z] + g[z & 1] * U[t][z];
                }
            }
            {
                uint32_t f[NM][4][4];
                to_frags<NM>(X, 1.0f, f);
                update_state<DK, NM, NT, false>(S, vec[V_GAM * kChunk + kChunk - 1], r_inv, f, kimg, f, kimg);
            }
            __syncwarp();
            if (lane == 0) umma::mbar_arrive(&ring.empty[st]);
            if (!SUMMARY && row0 < dv)
                store_transposed<T>(O, static_cast<T*>(a.out) + ((int64_t)w.sp.start + c * kChunk) * a.out_stride +
                                           (int64_t)w.head * dv + row0,
                                    a.out_stride, rows, dv - row0, mine + 2 * St::kRows);
        }
        if constexpr (!SUMMARY) {
            const bool again = __syncthreads_or(!(isfinite(S[0][0]) && isfinite(S[0][2])));      // of two rows
            if (again && !ring.dead) {
                redo_pass<T, DK, NM, NW, PASS>(a, smem);
                return;
            }
        }
        if (SUMMARY) {
            if (row0 < v_pad) {
                store_state(a.seg_state + (part + 1) * dv * dk, S, row0, dv, dk);
            } else {
                const float up = scale_up(tile_max(S));
                uint32_t f[2][KS][4];
                to_frags<2>(S, up, f);
                store_image<CG>(a.seg_map + part * 2 * DK * DK * 2, DK * DK * 2, f, (row0 - v_pad) / 8, CG);
                if (lane == 0) a.seg_unit[part * 8 + (row0 - v_pad) / 16] = pow2_inv(up);
            }
        } else if (a.last && w.seg == a.segments - 1) {
            store_state(a.last + states, S, row0, dv, dk);
        }
    }
    ring_end(a, ring, stages);
}

template <typename T, int DK, int NW>
__global__ void __launch_bounds__(NW * 32, min_ctas<NW>()) delta_reverse_kernel(const __grid_constant__ ChainArgs a) {
    constexpr int NM = sizeof(T) == 4 ? 2 : 1;
    using St = Stage<T, DK, NM, NW>;
    constexpr int NT = St::NT, CG = DK / 8, KS = DK / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Ring ring;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    const Work w = work_of(a, blockIdx.x, 1, NW * 16, 1, 1);
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.counter = 0;
    ring_init<NW>(ring);
    const int stages = a.stages;
    uint8_t* mine = smem + stages * St::kBytes + warp * St::kWarp;
    if (warp == 0)
        for (int n = 0; n < stages - 1; ++n) copy_chunk<St, DK, true>(a, w, smem, ring, n, n, -1);
    {
        const int dk = a.shape.k_dim, dv = a.shape.v_dim, hv = a.shape.v_heads;
        const int row0 = warp * 16;
        const int64_t states = ((int64_t)w.e * hv + w.head) * dv * dk;
        float S[DK / 8][4];
        copy_rows<St, T>(a, w, mine, w.chunks - 1, row0);
        load_state(a.first ? a.first + states : nullptr, S, row0, dv, dk);
        int st = stages - 1, turn = -1;      // of the chunk before
        for (int n = 0; n < w.chunks; ++n) {
            const int c = w.chunks - 1 - n, st_before = st, turn_before = turn;
            if (++st == stages) st = 0, ++turn;
            copy_rows<St, T>(a, w, mine + ((n + 1) & 1) * St::kRows, c - 1, row0);
            if (stages == 1 && warp == 0) copy_chunk<St, DK, true>(a, w, smem, ring, n, 0, n - 1);
            stage_ready(ring, st, turn);
            const uint8_t* s = smem + st * St::kBytes;
            const uint32_t kimg = umma::smem_u32(s), qimg = kimg + NT * St::kKey, pair = kimg + St::kKeys;
            const float* vec = reinterpret_cast<const float*>(s + St::kKeys + 2 * kSquare);
            const int rows = min(kChunk, w.sp.len - c * kChunk);
            const int64_t at = (w.slot0 + c) * hv + w.head;
            if (stages > 1 && warp == 0)
                copy_chunk<St, DK, true>(a, w, smem, ring, n + stages - 1, st_before, turn_before);
            float U[8][4];
            zero(U);
            const float s_up = scale_up(across<NW>(ring, 0, tile_max(S))), s_inv = pow2_inv(s_up);
            {
                uint32_t f[NM][KS][4];
                to_frags<NM>(S, s_up, f);
                gemm<KS, 8, NM, NT, false>(U, f, kimg, St::kKey, CG, 0);
                const int64_t plane = (int64_t)NW * 16 * DK * 2;
                store_image<NT == 1 ? 1 : kSliceCols / 8>(a.state_img + at * NT * plane, plane, f, row0 / 8, NW * 2);
                if (threadIdx.x == 0) a.state_unit[at] = s_inv;
            }
            float dO[8][4];       // dout scale kq
            rows_ready();
            load_transposed<T, St::kPitch>(mine + (n & 1) * St::kRows, dO);
            mask_rows(dO, rows, dv - row0);
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const float2 qs = vec2(vec, V_QS, t);
#pragma unroll
                for (int z = 0; z < 4; ++z) dO[t][z] *= z & 1 ? qs.y : qs.x;
            }
            {
                const float up = scale_up(tile_max(dO)), inv = pow2_inv(up) * vec[V_MISC * kChunk + kPUnit];
                uint32_t f[NM][4][4];
                to_frags<NM>(dO, up, f);
                float d[8][4];
                zero(d);
                gemm<4, 8, NM, NM, true, kLower>(d, f, pair + kSquare, (int)kPairFirst, 8, 0);
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    const float2 r = vec2(vec, V_REST, t);
                    const float f2[2] = {r.x * s_inv, r.y * s_inv};
#pragma unroll
                    for (int z = 0; z < 4; ++z) U[t][z] = f2[z & 1] * U[t][z] + inv * d[t][z];
                }
            }
            float R[8][4];
            zero(R);
            {
                const float up = scale_up(tile_max(U)), inv = pow2_inv(up);
                uint32_t f[NM][4][4];
                to_frags<NM>(U, up, f);
                gemm<4, 8, NM, NM, false, kLower>(R, f, pair, (int)kPairFirst, 8, 0);
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    const float2 ti = vec2(vec, V_TINV, t);
                    const float f2[2] = {ti.x * inv, ti.y * inv};
#pragma unroll
                    for (int z = 0; z < 4; ++z) R[t][z] *= f2[z & 1];
                }
            }
            {
                const float up = scale_up(across<NW>(ring, 1, tile_max(R)));
                uint32_t f[NT][4][4];
                to_frags<NT>(R, up, f);
                const int64_t plane = (int64_t)NW * 16 * kChunk * 2;
                store_image<NT == 1 ? 1 : 8>(a.vec_img + at * NT * plane, plane, f, row0 / 8, NW * 2);
                if (threadIdx.x == 0) a.vec_unit[at] = pow2_inv(up);
            }
            // dv in R; gamma dO and -gamma dv^ for the state
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const float2 g = vec2(vec, V_GAM, t), dvf = vec2(vec, V_DV, t), dsf = vec2(vec, V_DS, t);
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    dO[t][z] *= z & 1 ? g.y : g.x;
                    U[t][z] = -R[t][z] * (z & 1 ? dsf.y : dsf.x);
                    R[t][z] *= z & 1 ? dvf.y : dvf.x;
                }
            }
            {
                const float up = scale_up(fmaxf(tile_max(dO), tile_max(U))), inv = pow2_inv(up);
                uint32_t f[NM][4][4], g[NM][4][4];
                to_frags<NM>(dO, up, f);
                to_frags<NM>(U, up, g);
                update_state<DK, NM, NT, true>(S, vec[V_GAM * kChunk + kChunk - 1], inv, f, qimg, g, kimg);
            }
            __syncwarp();
            if (lane == 0) umma::mbar_arrive(&ring.empty[st]);
            if (row0 < dv)
                store_transposed<T>(R, static_cast<T*>(a.out) + ((int64_t)w.sp.start + c * kChunk) * a.out_stride +
                                           (int64_t)w.head * dv + row0,
                                    a.out_stride, rows, dv - row0, mine + 2 * St::kRows);
        }
        if (a.last) store_state(a.last + states, S, row0, dv, dk);
    }
    ring_end(a, ring, stages);
}

// The parts' starts from their summaries, in order: S_{g+1} = S_g M_g + B_g,
// where seg_state holds B_g at g + 1 before and S_{g+1} after.  A chain of one
// product per part, so a CTA takes few rows and splits the columns: warp w
// makes columns w DK / 4 .. of 16 rows, and the rows come together again
// through shared memory.  M_g's two planes are copied a part ahead.  Bound by the
// latency of a step, 2 us: 19 parts of four heads of 128 x 128 36 us.
template <int DK>
struct Join {
    static constexpr int kMap = 2 * DK * DK * 2;
    static constexpr int kPitch = DK + 8;      // floats
    static constexpr int kShared = 2 * kMap + 16 * kPitch * 4;
};
template <int DK>
__global__ void __launch_bounds__(128) delta_join_kernel(const __grid_constant__ ChainArgs a) {
    constexpr int CG = DK / 8, KS = DK / 16, NT = DK / 32, P = Join<DK>::kPitch;
    extern __shared__ __align__(128) uint8_t smem[];
    float* rows = reinterpret_cast<float*>(smem + 2 * Join<DK>::kMap);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row4 = lane >> 2, col2 = (lane & 3) * 2;
    const int dk = a.shape.k_dim, dv = a.shape.v_dim;
    const int slices = (dv + 15) / 16;
    const int64_t item = blockIdx.x / slices;      // episode and head
    const int row0 = blockIdx.x % slices * 16;
    auto copy = [&](int g) {
        if (g < a.segments - 1) {
            const uint8_t* from = a.seg_map + (item * a.segments + g) * Join<DK>::kMap;
            const uint32_t to = umma::smem_u32(smem) + (g & 1) * Join<DK>::kMap;
            for (int i = threadIdx.x * 16; i < Join<DK>::kMap; i += 128 * 16)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i), "l"(from + i) : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // this warp's tiles of a state: rows row4, row4 + 8, columns (warp NT + t) 8 + col2
    auto load = [&](int g, float (&x)[NT][4]) {
        const float* from = a.seg_state + (item * a.segments + g) * dv * dk;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = row0 + row4 + 8 * h, c = (warp * NT + t) * 8 + col2;
                float2 v = make_float2(0.0f, 0.0f);
                if (r < dv && c < dk) v = *reinterpret_cast<const float2*>(from + (int64_t)r * dk + c);
                x[t][2 * h] = v.x;
                x[t][2 * h + 1] = v.y;
            }
    };
    auto share = [&](const float (&x)[NT][4]) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<float2*>(rows + (row4 + 8 * h) * P + (warp * NT + t) * 8 + col2) =
                    make_float2(x[t][2 * h], x[t][2 * h + 1]);
    };
    pdl_trigger();
    pdl_wait();
    copy(1);
    float N[NT][4];
    load(1, N);
    share(N);
    load(2, N);
    for (int g = 1; g < a.segments - 1; ++g) {
        copy(g + 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();
        const float* unit = a.seg_unit + (item * a.segments + g) * 8;
        float S[DK / 8][4];
#pragma unroll
        for (int t = 0; t < DK / 8; ++t) {      // the maps' units belong to their rows, S's columns
            const float u = unit[t / 2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float2 v = *reinterpret_cast<const float2*>(rows + (row4 + 8 * h) * P + t * 8 + col2);
                S[t][2 * h] = v.x * u;
                S[t][2 * h + 1] = v.y * u;
            }
        }
        const float up = scale_up(tile_max(S)), inv = pow2_inv(up);
        uint32_t f[2][KS][4];
        to_frags<2>(S, up, f);
        float d[NT][4];
        zero(d);
        gemm<KS, NT, 2, 2, true>(d, f, umma::smem_u32(smem) + (g & 1) * Join<DK>::kMap, DK * DK * 2, CG, warp * NT);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int z = 0; z < 4; ++z) d[t][z] = N[t][z] + inv * d[t][z];
        if (g + 2 < a.segments) load(g + 2, N);
        float* to = a.seg_state + (item * a.segments + g + 1) * dv * dk;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = row0 + row4 + 8 * h, c = (warp * NT + t) * 8 + col2;
                if (r < dv && c < dk)
                    *reinterpret_cast<float2*>(to + (int64_t)r * dk + c) = make_float2(d[t][2 * h], d[t][2 * h + 1]);
            }
        __syncthreads();
        share(d);
    }
}

template <auto KERNEL>
cudaError_t go(int nw, int smem, int most, int per_head, const ChainArgs& c, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    const int64_t grid = (int64_t)c.episodes * c.shape.v_heads * per_head;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    const cudaError_t e = opt_in(KERNEL, most, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(KERNEL, dim3((unsigned)grid), dim3(nw * 32), smem, st, c);
}

// Whether one stage is enough for a pass whose ring would keep a second CTA off
// the SM: where there are CTAs for more than one on each, and either no more than
// two (else a second round begins), or episodes of one chunk, which has nothing
// to copy ahead.  Read / one stage, us: 1000 heads of 30 tokens of 128 x 64,
// bf16, 55.1 / 47.0; 240 heads of 500 89.7 / 82.0; 160 of 300 of 64 x 64, fp32,
// 64.2 / 54.9; but 400 heads of 300 tokens 90.3 / 94.3, 120 of 200 33.7 / 36.3.
bool one_stage(const ChainArgs& c, int64_t grid, int num_sms) {
    return grid > num_sms && c.segments == 1 && (grid <= 2LL * num_sms || c.in.tokens <= (int64_t)kChunk * c.episodes);
}

// A pass over chunks with its ring.
template <auto KERNEL, typename St, int NW>
cudaError_t go_ring(int per_head, ChainArgs c, int num_sms, cudaStream_t st) {
    constexpr int kOne = St::kBytes + NW * St::kWarp;
    const int64_t grid = (int64_t)c.episodes * c.shape.v_heads * per_head;
    const bool one = NW == 4 && St::kShared > 112 * 1024 && kOne <= 112 * 1024 && one_stage(c, grid, num_sms);
    c.stages = one ? 1 : St::kCount;
    return go<KERNEL>(NW, one ? kOne : St::kShared, St::kShared, per_head, c, st);
}

template <typename T, int DK, int NM>
cudaError_t forward(const ChainArgs& c, int num_sms, cudaStream_t st) {
    using S4 = Stage<T, DK, NM, 4>;
    using S8 = Stage<T, DK, NM, 8>;
    const int slices = (c.shape.v_dim + 63) / 64;
    if (c.state_img) {
        if constexpr (NM == 2)      // with one plane, more than 64 channels are on tcgen05
            if (c.shape.v_dim > 64) return go_ring<delta_forward_kernel<T, DK, NM, 8, kSave>, S8, 8>(1, c, num_sms, st);
        return go_ring<delta_forward_kernel<T, DK, NM, 4, kSave>, S4, 4>(1, c, num_sms, st);
    }
    if (c.segments > 1) {
        cudaError_t e = go_ring<delta_forward_kernel<T, DK, NM, 4, kSummary>, S4, 4>(
            (slices + DK / 64) * (c.segments - 1), c, num_sms, st);
        if (e == cudaSuccess && c.segments > 2)
            e = go<delta_join_kernel<DK>>(4, Join<DK>::kShared, Join<DK>::kShared, (c.shape.v_dim + 15) / 16, c, st);
        if (e != cudaSuccess) return e;
    }
    // More than 64 channels: two CTAs of four warps per head, or one of eight,
    // which reads keys and pairs once, where heads alone fill the SMs (bf16 with
    // one plane is on tcgen05 then).  400 heads of 300 tokens of 128 x 128, fp32:
    // 330 us against 275; 462 ragged ones of 40 x 72 126 against 108; 80 heads
    // of 64 x 96 87 against 88.
    if constexpr (NM == 2)
        if (c.segments == 1 && c.shape.v_dim > 64 && (int64_t)c.episodes * c.shape.v_heads >= num_sms)
            return go_ring<delta_forward_kernel<T, DK, NM, 8, kOutputs>, S8, 8>(1, c, num_sms, st);
    return go_ring<delta_forward_kernel<T, DK, NM, 4, kOutputs>, S4, 4>(slices * c.segments, c, num_sms, st);
}
template <typename T, int DK>
cudaError_t reverse(const ChainArgs& c, int num_sms, cudaStream_t st) {
    constexpr int NM = sizeof(T) == 4 ? 2 : 1;
    if constexpr (NM == 2)
        if (c.shape.v_dim > 64) return go_ring<delta_reverse_kernel<T, DK, 8>, Stage<T, DK, NM, 8>, 8>(1, c, num_sms, st);
    return go_ring<delta_reverse_kernel<T, DK, 4>, Stage<T, DK, NM, 4>, 4>(1, c, num_sms, st);
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
    c.segments = 1;
    c.seg_state = nullptr;
    c.seg_map = nullptr;
    c.seg_unit = nullptr;
    c.counter = a.counter;
    c.status = a.status;
    return c;
}

}  // namespace

// Whether a pass fills tcgen05's 128 rows: more than 64 value channels, and
// operands of one plane (two do not fit in shared memory).  With 64 channels
// or fewer half the rows would be empty: a chunk takes a CTA 4.4 us there
// however many rows are filled, against 3 us for four warps of mma.sync that
// hold 64 channels' state in registers.  About 65k ragged transitions, four
// heads of 128 x 128, forward and reverse: 143 + 162 us, on mma.sync 197 + 206.
bool rows_of_tcgen05(const ofrl_delta_shape& s) { return s.dtype == OFRL_DTYPE_BF16 && s.v_dim > 64; }

// A forward pass that saves nothing has less to convert, and where two CTAs per
// head still find an SM each, mma.sync on 64 channels in each is the faster one:
// 32 heads of 2000 tokens of 128 x 128 118 us against 131, 64 heads of 512 40.3
// against 44.4; but 256 heads of 64 tokens 31.8 against 25.4, 400 of 300 143
// against 107.
bool forward_on_tcgen05(const SeqLaunch& a) {
    return rows_of_tcgen05(a.shape) && (a.saved || 2LL * a.episodes * a.shape.v_heads > a.num_sms);
}

// CTAs of the forward pass that share an SM.
template <typename T, int DK, int NM>
constexpr int together() { return Stage<T, DK, NM, 4>::kShared <= 112 * 1024 ? 2 : 1; }
int forward_together(const ofrl_delta_shape& s, int planes) {
    const bool wide = s.k_dim > 64;
    if (s.dtype == OFRL_DTYPE_F32) return wide ? together<float, 128, 2>() : together<float, 64, 2>();
    if (planes == 2) return wide ? together<__nv_bfloat16, 128, 2>() : together<__nv_bfloat16, 64, 2>();
    return wide ? together<__nv_bfloat16, 128, 1>() : together<__nv_bfloat16, 64, 1>();
}

// Parts of an episode.  A forward pass takes one CTA per head and 64 value
// channels; where these leave most SMs idle and episodes are long, each is cut
// into parts: summaries of all parts at once, the short chain over them, then
// all parts at once.  That is about 1.7 times the work and a step of the chain
// over parts costs about 0.4 chunks' time, so n chunks in g parts take about
// 1.7 n / g + 0.4 g instead of n; g = 2 sqrt(n) is best, but no more than the
// SMs hold at once in the last pass (a few CTAs more would be a second round).
// One sequence of 32768 tokens, four heads of 128, with its final state: 2100 us
// whole, 350 in 19 parts, in 20 (160 CTAs on 152 SMs) 65 more.  Three of 1000 tokens,
// two heads of 64, fp32: 73 us whole, 38 in 7 parts of 3 chunks, 33 in 8 of 2.
int segments_of(const SeqLaunch& a, int planes) {
    const int64_t items = (int64_t)a.episodes * a.shape.v_heads;
    const int slices = (a.shape.v_dim + 63) / 64;
    const double chunks = (double)a.in.tokens / kChunk / a.episodes;
    const int64_t room = (int64_t)forward_together(a.shape, planes) * a.num_sms / (items * slices);
    if (room < 4 || chunks < 12.0) return 1;
    // whole chunks to a part
    const double part = std::max(std::round(0.5 * std::sqrt(chunks)), std::ceil(chunks / (double)room));
    const int g = (int)std::ceil(chunks / part);
    return g >= 4 ? g : 1;
}

cudaError_t launch_chain_forward(const SeqLaunch& a, const Prepared& p, const Images& img, int planes, cudaStream_t st) {
    ChainArgs c = base_args(a, p, img);
    if (!a.saved) {
        c.segments = segments_of(a, planes);
        const int dkp = pad_dim(a.shape.k_dim);
        const int64_t parts = (int64_t)a.episodes * a.shape.v_heads * c.segments;
        uint8_t* at = a.parts;
        c.seg_state = reinterpret_cast<float*>(at);
        at += (parts * a.shape.v_dim * a.shape.k_dim * 4 + 255) / 256 * 256;
        c.seg_map = at;
        c.seg_unit = reinterpret_cast<float*>(at + parts * 2 * dkp * dkp * 2);
    }
    c.first = a.init;
    c.last = a.final_state;
    c.out = a.out;
    c.out_stride = (int64_t)a.shape.v_heads * a.shape.v_dim;
    c.rows = a.in.v;
    c.row_stride = a.in.v_stride;
    if (forward_on_tcgen05(a) && planes == 1 && c.segments == 1) return launch_chain_forward_tc(a, p, img, st);
    const bool wide = a.shape.k_dim > 64;
    const int sms = a.num_sms;
    if (a.shape.dtype == OFRL_DTYPE_F32) return wide ? forward<float, 128, 2>(c, sms, st) : forward<float, 64, 2>(c, sms, st);
    if (planes == 2) return wide ? forward<__nv_bfloat16, 128, 2>(c, sms, st) : forward<__nv_bfloat16, 64, 2>(c, sms, st);
    return wide ? forward<__nv_bfloat16, 128, 1>(c, sms, st) : forward<__nv_bfloat16, 64, 1>(c, sms, st);
}

cudaError_t launch_chain_reverse(const SeqLaunch& a, const Prepared& p, const Images& img, cudaStream_t st) {
    if (rows_of_tcgen05(a.shape)) return launch_chain_reverse_tc(a, p, img, st);
    ChainArgs c = base_args(a, p, img);
    c.first = a.d_final;
    c.last = a.d_init;
    c.out = a.grads.dv;
    c.out_stride = a.grads.v_stride;
    c.rows = a.dout;
    c.row_stride = (int64_t)a.shape.v_heads * a.shape.v_dim;
    const bool wide = a.shape.k_dim > 64;
    if (a.shape.dtype == OFRL_DTYPE_F32) return wide ? reverse<float, 128>(c, a.num_sms, st) : reverse<float, 64>(c, a.num_sms, st);
    return wide ? reverse<__nv_bfloat16, 128>(c, a.num_sms, st) : reverse<__nv_bfloat16, 64>(c, a.num_sms, st);
}

}  // namespace delta
}  // namespace ofrl
