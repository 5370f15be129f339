// Shared declarations of the selective scan's kernels and their context.
//
// Per channel d and state n (A2 = A log2 e, so that exp is exp2):
//   h_t = a_t h_{t-1} + delta_t B_t x_t,  a_t = exp2(delta_t A2),  y_t = sum_n C_t h_t.
//
// The packed tokens are cut into segments of equal length, whatever the
// episodes are; a segment is one CTA's for a block of channels, and the state
// is reset inside it where an episode begins.  What a segment needs from the
// ones before it is the state its first token continues:
//   1. scan_tail_kernel: the state each segment ends with, from the last start
//      of an episode within it (or from zero, with the sum of its deltas)
//   2. scan_carry_kernel: those joined over the segments,
//      carry <- exp2(A2 sum delta) carry + tail
//   3. the segments themselves
// A segment whose successor begins an episode has no tail, so packed short
// episodes cost nearly nothing in 1.  The gradients run the same three steps
// from the other end.  The segments depend on the sizes alone, so results do not
// depend on what runs beside.
#pragma once

#include "episodes.cuh"
#include "lanes.cuh"

struct ofrl_scan {
    int device;
    int num_sms;
    ofrl_scan_shape shape;
    int64_t max_tokens;
    int32_t max_episodes;
    int32_t backward;
    void* base;          // the single cudaMalloc of the context
    int64_t bytes;
    int32_t* status;     // [OFRL_STAT_WORDS]
    uint8_t* work;       // what lies between the launches of one call
};

namespace ofrl {
namespace scan {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kTile = 16;            // tokens brought into shared memory at once
constexpr int kSave = 8;             // tokens between saved states: a tile of the gradients
constexpr int kMaxSegment = 4096;    // tokens of a segment (its mask of starts is in shared memory)
constexpr int kMinSegment = 64;

// How a state of [channels, N] lies on a warp: LS lanes share a channel, four
// states each, and a thread has CPT channels.
constexpr int lanes_of(int n) { return n <= 4 ? 1 : n <= 8 ? 2 : n <= 16 ? 4 : n <= 32 ? 8 : 16; }
// CPT of a call's two forms, the wide one and the one for little work.
constexpr int wide_of(int ls) { return ls < 2 ? 1 : ls < 4 ? 2 : 4; }
constexpr int narrow_of(int ls, bool backward) { return backward && ls >= 4 ? 2 : 1; }
constexpr int block_of(int ls, int cpt) { return kWarps * (32 / ls) * cpt; }      // channels of a CTA

// How one call is cut.
struct Cut {
    int ls, cpt;
    int blocks;          // CTAs over the channels, all groups
    int seg;             // tokens of a segment
    int n_seg;           // at least 1
};
Cut cut_of(const ofrl_scan_shape& s, int64_t tokens, int64_t episodes, int num_sms, bool backward);

// Bytes from the workspace's start.
struct Work {
    int64_t tail;        // [n_seg][channels][N] tails, then carries
    int64_t sum;         // [n_seg][channels] sums of delta
    int64_t kind;        // [n_seg] Tail
    int64_t dbc;         // backward: [blocks of a group][tokens][groups][2 NP] parts of dB and dC
    int64_t da;          // backward: [n_seg][channels][N]
    int64_t dd;          // backward: [n_seg][channels] of dD, then of ddt_bias
    int64_t total;
};
Work work_of(const ofrl_scan_shape& s, int64_t tokens, const Cut& c, bool backward);
int64_t work_bytes(const ofrl_scan_shape& s, int64_t max_tokens, int num_sms, bool backward);

// What a segment hands on.
enum Tail : int32_t {
    kTailNone = 0,       // the next segment begins an episode: nothing
    kTailOwn = 1,        // its tail alone
    kTailJoin = 2        // its tail and what it took over, decayed
};

struct Launch {
    ofrl_scan_shape shape;
    ofrl_scan_tokens in;
    const int32_t* ends;
    int32_t episodes;
    const float* init;
    void* out;
    int64_t out_stride;
    float* final_state;
    float* saved;        // [tokens / kSave][channels][N]
    const void* dout;
    int64_t dout_stride;
    const float* d_final;
    ofrl_scan_grads grads;
    float* d_init;
    int32_t* status;
    float* tail;
    float* sum;
    int32_t* kind;
    float* dbc;
    float* da;
    float* dd;
    int seg, n_seg, blocks;     // of the Cut
};

struct StepLaunch {
    ofrl_scan_shape shape;
    ofrl_scan_tokens in;
    const int32_t* slot_idx;
    int32_t slots;
    const float* state_in;
    float* state_out;
    void* out;
    int64_t out_stride;
    int32_t* status;
    int num_sms;
    int whole_states;    // B and C can be read four elements at a time
};

cudaError_t launch_forward(const Launch& a, const Cut& c, cudaStream_t st);
cudaError_t launch_backward(const Launch& a, const Cut& c, cudaStream_t st);
cudaError_t launch_carry(const Launch& a, bool backward, cudaStream_t st);
cudaError_t launch_step(const StepLaunch& a, cudaStream_t st);
int64_t saved_bytes(const ofrl_scan_shape& s, int64_t tokens);

// ---- what a CTA holds -------------------------------------------------------------

// How the CTA's threads take a tile [ROWS tokens][CB channels] of a row buffer:
// vectors of V elements, NV a thread, always in the same column.
template <typename T, int CB, int ROWS>
struct Tiling {
    static constexpr int kEach = ROWS * CB / kThreads;
    // gradients: four, whose fp32 forms threads write side by side without conflicts
    static constexpr int kMost = ROWS < kTile ? 4 : 16 / (int)sizeof(T);
    static constexpr int V = kEach < 1 ? 1 : kEach < kMost ? kEach : kMost;
    static constexpr int NV = kEach < V ? 1 : kEach / V;
    static constexpr int kCols = CB / V;             // threads along a row
    static constexpr int kRowStep = kThreads / kCols;
    static_assert(CB % V == 0 && kThreads % kCols == 0, "a thread stays in its column");
    __device__ static int col() { return (int)threadIdx.x % kCols * V; }
    __device__ static int row(int j) { return (int)threadIdx.x / kCols + j * kRowStep; }
};

// The CTA's channels.
struct Block {
    int group, ch0, count;      // first channel (of all) and how many
};
__device__ __forceinline__ Block block_at(const ofrl_scan_shape& s, int blocks, int cb, int y) {
    const int per_group = s.channels / s.groups, n = blocks / s.groups;
    Block b;
    b.group = y / n;
    const int at = (y - b.group * n) * cb;
    b.ch0 = b.group * per_group + at;
    b.count = min(cb, per_group - at);
    return b;
}

// One token's operands of a thread, and the pairs its states make.  With CPT
// >= 2 a pair is two channels of one state, so that what belongs to channels
// (delta, x, dy) lies in pairs as it is and what belongs to states (B, C) is
// stored twice; with one channel a pair is two states of it.
template <int LS, int CPT>
struct Lay {
    static constexpr bool kWide = CPT >= 2;
    static constexpr int kPairs = 2 * CPT;
    static constexpr int kCh = kWide ? CPT / 2 : 1;       // channel operands
    static constexpr int kSt = kWide ? 4 : 2;             // state operands
    static constexpr int NP = 4 * LS;
    static constexpr int kStWidth = kWide ? 2 * NP : NP;  // floats of a token's B in shared memory
    static constexpr int CW = 32 / LS * CPT, CB = kWarps * CW;
    __device__ static constexpr int ci(int q) { return kWide ? q / 4 : 0; }
    __device__ static constexpr int si(int q) { return kWide ? q % 4 : q; }

    // channel operands from a tile's row (at the thread's first channel)
    __device__ static void channels(f2 (&o)[kCh], const float* p) {
        if constexpr (CPT == 4) {
            const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(p);
            o[0] = u.x;
            o[1] = u.y;
        } else if constexpr (CPT == 2) {
            o[0] = *reinterpret_cast<const f2*>(p);
        } else {
            o[0] = f2_of(*p, *p);
        }
    }
    // state operands from a token's B or C (at the thread's first state)
    __device__ static void states(f2 (&o)[kSt], const float* p) {
#pragma unroll
        for (int i = 0; i < kSt / 2; ++i) {
            const ulonglong2 u = reinterpret_cast<const ulonglong2*>(p)[i];
            o[2 * i] = u.x;
            o[2 * i + 1] = u.y;
        }
    }
    // where a thread's states operands begin in a token's B
    __device__ static int state_at(int ls) { return kWide ? 8 * ls : 4 * ls; }
    // a thread's states [CPT channels][4] <-> its pairs
    __device__ static f2 pair_of(const float (&v)[CPT][4], int q) {
        if constexpr (kWide)
            return f2_of(v[2 * ci(q)][si(q)], v[2 * ci(q) + 1][si(q)]);
        else
            return f2_of(v[0][2 * q], v[0][2 * q + 1]);
    }
    __device__ static void unpair(float (&v)[CPT][4], const f2 (&h)[kPairs]) {
#pragma unroll
        for (int q = 0; q < kPairs; ++q) {
            if constexpr (kWide)
                f2_split(h[q], v[2 * ci(q)][si(q)], v[2 * ci(q) + 1][si(q)]);
            else
                f2_split(h[q], v[0][2 * q], v[0][2 * q + 1]);
        }
    }
};

// A thread's states of [.., channels, N] fp32 rows: loads (zero where it has
// none) and stores.  base: row of channel 0.
template <int LS, int CPT>
__device__ __forceinline__ void load_states(f2 (&h)[2 * CPT], const float* base, int n, int ch, int count, int n0) {
    float v[CPT][4];
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
        float4 u = make_float4(0, 0, 0, 0);
        if (i < count && n0 < n) u = *reinterpret_cast<const float4*>(base + (int64_t)(ch + i) * n + n0);
        v[i][0] = u.x;
        v[i][1] = u.y;
        v[i][2] = u.z;
        v[i][3] = u.w;
    }
#pragma unroll
    for (int q = 0; q < 2 * CPT; ++q) h[q] = Lay<LS, CPT>::pair_of(v, q);
}
template <int LS, int CPT>
__device__ __forceinline__ void store_states(float* base, const f2 (&h)[2 * CPT], int n, int ch, int count, int n0) {
    float v[CPT][4];
    Lay<LS, CPT>::unpair(v, h);
#pragma unroll
    for (int i = 0; i < CPT; ++i)
        if (i < count && n0 < n)
            *reinterpret_cast<float4*>(base + (int64_t)(ch + i) * n + n0) =
                make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
}

__device__ __forceinline__ f2 delta_of(f2 dt, f2 bias, int with_softplus) {
    const f2 v = f2_add(dt, bias);
    return with_softplus ? softplus(v) : v;
}

// Elements i and i + 1 of a thread's V (one element stands twice).
template <int V>
__device__ __forceinline__ f2 pair_at(const float (&x)[V], int i) {
    return f2_of(x[i], x[V > 1 ? i + 1 : i]);
}
template <int V>
__device__ __forceinline__ void set_pair(float (&x)[V], int i, f2 v) {
    x[i] = f2_lo(v);
    if constexpr (V > 1) x[i + 1] = f2_hi(v);
}

// Sums over the LS lanes of a channel.  Wide forms hand the channels out: the
// first min(CPT, LS) lanes return one channel each (channel `which`).
template <int LS, int CPT>
__device__ __forceinline__ int which_channel() {
    const int lane = threadIdx.x & 31;
    if constexpr (CPT == 4)
        return (lane & 1) * 2 + ((lane >> 1) & 1);
    else if constexpr (CPT == 2)
        return lane & 1;
    else
        return 0;
}
// 1 in the lanes that return a channel's sum.
template <int LS, int CPT>
__device__ __forceinline__ bool returns_channel() {
    const int ls = (threadIdx.x & 31) % LS;
    return ls < CPT;
}
template <int LS, int CPT>
__device__ __forceinline__ float sum_states(const float (&y)[CPT]) {
    const int lane = threadIdx.x & 31;
    float r;
    if constexpr (CPT == 4) {
        static_assert(LS >= 4, "");
        const bool up = lane & 1;
        float a = up ? y[2] : y[0], b = up ? y[3] : y[1];
        a += __shfl_xor_sync(0xffffffffu, up ? y[0] : y[2], 1);
        b += __shfl_xor_sync(0xffffffffu, up ? y[1] : y[3], 1);
        const bool up2 = lane & 2;
        r = (up2 ? b : a) + __shfl_xor_sync(0xffffffffu, up2 ? a : b, 2);
#pragma unroll
        for (int o = 4; o < LS; o <<= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
    } else if constexpr (CPT == 2) {
        static_assert(LS >= 2, "");
        const bool up = lane & 1;
        r = (up ? y[1] : y[0]) + __shfl_xor_sync(0xffffffffu, up ? y[0] : y[1], 1);
#pragma unroll
        for (int o = 2; o < LS; o <<= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
    } else {
        r = y[0];
#pragma unroll
        for (int o = 1; o < LS; o <<= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
    }
    return r;
}

// V floats to shared memory (V-aligned).
template <int V>
__device__ __forceinline__ void put_floats(float* dst, const float (&x)[V]) {
    if constexpr (V == 8) {
        reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        store_vec<float, V>(dst, x);
    }
}

// A row buffer as a CTA goes along it: the thread's first vector of a tile, and how
// far apart its vectors are.
template <typename T, int CB, int ROWS = kTile>
struct Rows {
    using Ti = Tiling<T, CB, ROWS>;
    const T* p;
    int64_t stride, apart;
    bool on;
    __device__ Rows(const void* src, int64_t stride_, const Block& b, int t0) {
        stride = stride_;
        apart = Ti::kRowStep * stride;
        on = Ti::col() < b.count;
        p = static_cast<const T*>(src) + (int64_t)(t0 + Ti::row(0)) * stride + b.ch0 + Ti::col();
    }
    __device__ void move(int tiles) { p += tiles * ROWS * stride; }
};

// A tile of one row buffer in shared memory, as it came: every thread copies what
// it reads itself, so it has to wait for its own copies only.
template <typename T, int CB>
struct RowsCopied {
    using Ti = Tiling<T, CB, kTile>;
    Vec<T, Ti::V> v[Ti::NV][kThreads];
    // once: vectors past the CTA's channels stay zero
    __device__ void clear() {
#pragma unroll
        for (int j = 0; j < Ti::NV; ++j)
#pragma unroll
            for (int i = 0; i < Ti::V; ++i) v[j][threadIdx.x].v[i] = from_float<T>(0.0f);
    }
    __device__ void ask(const Rows<T, CB>& from, int rows) {
        constexpr int kBytes = Ti::V * (int)sizeof(T);
#pragma unroll
        for (int j = 0; j < Ti::NV; ++j) {
            if (!from.on || Ti::row(j) >= rows) continue;
            if constexpr (kBytes >= 4)
                copy_async<kBytes>(&v[j][threadIdx.x], from.p + j * from.apart);
            else
                v[j][threadIdx.x] = *reinterpret_cast<const Vec<T, Ti::V>*>(from.p + j * from.apart);
        }
    }
    __device__ Vec<T, Ti::V> at(int j) const { return v[j][threadIdx.x]; }
};
// Elements i and i + 1 of a vector (one element stands twice).
template <typename T, int V>
__device__ __forceinline__ f2 pair_of(const Vec<T, V>& u, int i) {
    if constexpr (V > 1)
        return vec_pair(u, i / 2);
    else
        return f2_both(to_float(u.v[0]));
}

// A tile of one row buffer on its way in registers.  The loads stay where they
// are asked for: the compiler would move them to their use.
template <typename T, int CB, int ROWS>
struct RowsHeld {
    using Ti = Tiling<T, CB, ROWS>;
    Vec<T, Ti::V> v[Ti::NV];
    __device__ void ask(const Rows<T, CB, ROWS>& from, int rows) {
#pragma unroll
        for (int j = 0; j < Ti::NV; ++j) {
#pragma unroll
            for (int i = 0; i < Ti::V; ++i) v[j].v[i] = from_float<T>(0.0f);
            if (!from.on || Ti::row(j) >= rows) continue;
            const T* src = from.p + j * from.apart;
            uint32_t* w = reinterpret_cast<uint32_t*>(&v[j]);
            if constexpr (sizeof(v[j]) == 16)
                asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(src) : "memory");
            else if constexpr (sizeof(v[j]) == 8)
                asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(src) : "memory");
            else if constexpr (sizeof(v[j]) == 4)
                asm volatile("ld.global.b32 %0, [%1];" : "=r"(w[0]) : "l"(src) : "memory");
            else
                v[j] = *reinterpret_cast<const Vec<T, Ti::V>*>(src);
        }
    }
    __device__ const Vec<T, Ti::V>& at(int j) const { return v[j]; }
};

// B or C of a tile, in flight.
template <typename T, int LS, int CPT, int ROWS = kTile>
struct StatesHeld {
    using L = Lay<LS, CPT>;
    static constexpr int kEach = ROWS * L::NP / kThreads < 1 ? 1 : ROWS * L::NP / kThreads;
    T v[kEach];
    __device__ void load(const void* src, int64_t stride, int group, int n, int t0, int rows) {
        const T* p = static_cast<const T*>(src) + group * n;
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int i = threadIdx.x + j * kThreads, r = i / L::NP, k = i % L::NP;
            v[j] = r < rows && k < n ? p[(int64_t)(t0 + r) * stride + k] : from_float<T>(0.0f);
        }
    }
    __device__ void put(float* dst) const {
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int i = threadIdx.x + j * kThreads, r = i / L::NP, k = i % L::NP;
            if (r >= ROWS) continue;
            const float x = to_float(v[j]);
            if constexpr (L::kWide)
                *reinterpret_cast<float2*>(dst + r * L::kStWidth + 2 * k) = make_float2(x, x);
            else
                dst[r * L::kStWidth + k] = x;
        }
    }
};

template <typename T, int CB, int ROWS>
__device__ __forceinline__ void load_params(float (&v)[Tiling<T, CB, ROWS>::V], const float* p, const Block& b) {
    using Ti = Tiling<T, CB, ROWS>;
#pragma unroll
    for (int i = 0; i < Ti::V; ++i) v[i] = p != nullptr && Ti::col() + i < b.count ? p[b.ch0 + Ti::col() + i] : 0.0f;
}

// The thread's place among the states.
template <int LS, int CPT>
struct Place {
    int local, ch, count, n0;     // first channel (in the CTA, of all), how many of them exist, first state
    __device__ Place(const Block& b) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        local = warp * Lay<LS, CPT>::CW + lane / LS * CPT;
        ch = b.ch0 + local;
        count = max(0, min(CPT, b.count - local));
        n0 = lane % LS * 4;
    }
};

template <int LS, int CPT>
__device__ __forceinline__ void load_decays(f2 (&a2)[2 * CPT], const Launch& a, const Place<LS, CPT>& p) {
    load_states<LS, CPT>(a2, a.in.a, a.shape.state_dim, p.ch, p.count, p.n0);
    const f2 k = f2_of(kLog2e, kLog2e);
#pragma unroll
    for (int q = 0; q < 2 * CPT; ++q) a2[q] = f2_mul(a2[q], k);
}

}  // namespace scan
}  // namespace ofrl
