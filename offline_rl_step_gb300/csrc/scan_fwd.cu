// Selective scan, forward: tails of segments, their join, the segments.

#include "scan.cuh"

namespace ofrl {
namespace scan {
namespace {

template <typename T, int LS, int CPT>
struct TailShared {
    using L = Lay<LS, CPT>;
    alignas(16) float delta[kTile][L::CB];
    alignas(16) float dx[kTile][L::CB];      // delta x
    alignas(16) float b[kTile * L::kStWidth];
    alignas(16) RowsCopied<T, L::CB> x, dt;
    uint32_t mask[kMaxSegment / 32];
    Range range;
};
template <typename T, int LS, int CPT>
struct ForwardShared {
    using L = Lay<LS, CPT>;
    alignas(16) float delta[kTile][L::CB];
    alignas(16) float dx[kTile][L::CB];      // delta x, then sum_n C h
    alignas(16) float b[kTile * L::kStWidth];
    alignas(16) float c[kTile * L::kStWidth];
    alignas(16) RowsCopied<T, L::CB> x[2], dt, z;
    uint32_t mask[kMaxSegment / 32];
    Range range;
};

// delta and delta x of a tile.
template <typename T, int CB>
__device__ __forceinline__ void put_rows(float (*delta)[CB], float (*dx)[CB], const RowsCopied<T, CB>& x,
                                         const RowsCopied<T, CB>& dt, const float (&bias)[Tiling<T, CB, kTile>::V],
                                         int with_softplus) {
    using Ti = Tiling<T, CB, kTile>;
#pragma unroll
    for (int j = 0; j < Ti::NV; ++j) {
        const int r = Ti::row(j);
        if (r >= kTile) continue;
        const Vec<T, Ti::V> xv = x.at(j), dv = dt.at(j);
        float d[Ti::V], u[Ti::V];
#pragma unroll
        for (int i = 0; i < Ti::V; i += 2) {
            const f2 de = delta_of(pair_of(dv, i), pair_at(bias, i), with_softplus);
            set_pair(d, i, de);
            set_pair(u, i, f2_mul(de, pair_of(xv, i)));
        }
        put_floats(&delta[r][Ti::col()], d);
        put_floats(&dx[r][Ti::col()], u);
    }
}

// 1. The state a segment ends with, as far as it is the segment's own.  The same
// steps as 3 without outputs: 32768 tokens of one episode, 1024 channels of 16
// states, bf16, 107 us beside its 166; 228 episodes of 64 to 512 tokens, 512
// channels, 105 beside 187 (the longest tail of a segment counts).
template <typename T, int LS, int CPT>
__global__ void __launch_bounds__(kThreads, 4) scan_tail_kernel(const __grid_constant__ Launch a) {
    using L = Lay<LS, CPT>;
    using Ti = Tiling<T, L::CB, kTile>;
    extern __shared__ __align__(16) uint8_t dynamic[];
    auto& s = *reinterpret_cast<TailShared<T, LS, CPT>*>(dynamic);
    pdl_wait();
    pdl_trigger();
    const int tokens = (int)a.in.tokens, n = a.shape.state_dim;
    const int s0 = (int)((int64_t)blockIdx.x * a.seg), s1 = (int)min((int64_t)s0 + a.seg, (int64_t)tokens);
    for (int i = threadIdx.x; i < kMaxSegment / 32; i += kThreads) s.mask[i] = 0;
    __syncthreads();
    if (threadIdx.x < 32) {
        const Range r = mark_starts(a.ends, a.episodes, tokens, s0, s1, s.mask);
        if (threadIdx.x == 0) s.range = r;
    }
    __syncthreads();
    if (s.range.closed) {
        if (threadIdx.x == 0 && blockIdx.y == 0) a.kind[blockIdx.x] = kTailNone;
        return;
    }
    int begin = s0, own = 0;
    for (int w = (s1 - s0 - 1) >> 5; w >= 0; --w)
        if (s.mask[w]) {
            begin = s0 + w * 32 + 31 - __clz(s.mask[w]);
            own = 1;
            break;
        }
    if (threadIdx.x == 0 && blockIdx.y == 0) a.kind[blockIdx.x] = own ? kTailOwn : kTailJoin;

    const Block b = block_at(a.shape, a.blocks, L::CB, blockIdx.y);
    const Place<LS, CPT> p(b);
    Rows<T, L::CB> x(a.in.x, a.in.x_stride, b, begin), dt(a.in.dt, a.in.dt_stride, b, begin);
    StatesHeld<T, LS, CPT> bs;
    auto fetch = [&](int t0) {      // the tile after the ones asked for
        const int rows = min(kTile, s1 - t0);
        s.x.ask(x, rows);
        s.dt.ask(dt, rows);
        copies_commit();
        bs.load(a.in.b, a.in.b_stride, b.group, n, t0, rows);
        x.move(1);
        dt.move(1);
    };
    s.x.clear();
    s.dt.clear();
    fetch(begin);
    f2 a2[L::kPairs], h[L::kPairs], sum[L::kCh];
    load_decays<LS, CPT>(a2, a, p);
    float bias[Ti::V];
    load_params<T, L::CB, kTile>(bias, a.in.dt_bias, b);
#pragma unroll
    for (int i = 0; i < L::kCh; ++i) sum[i] = f2_of(0.0f, 0.0f);
#pragma unroll
    for (int q = 0; q < L::kPairs; ++q) h[q] = f2_of(0.0f, 0.0f);
    if (own && a.init != nullptr) {
        const int e = find_episode(a.ends, s.range.e0, a.episodes, tokens, s1 - 1);
        load_states<LS, CPT>(h, a.init + (int64_t)min(e, a.episodes - 1) * a.shape.channels * n, n, p.ch, p.count, p.n0);
    }
    for (int t0 = begin; t0 < s1; t0 += kTile) {
        const int rows = min(kTile, s1 - t0);
        copies_wait<0>();
        __syncthreads();      // the tile before is through
        put_rows(s.delta, s.dx, s.x, s.dt, bias, a.shape.softplus);
        bs.put(s.b);
        __syncthreads();
        if (t0 + kTile < s1) fetch(t0 + kTile);
        // the tile's deltas, from zero: one running sum over a segment rounds steps that hardly change
        // the same way for thousands of tokens (4096 of them 6e-5 off)
        f2 steps[L::kCh];
#pragma unroll
        for (int k = 0; k < L::kCh; ++k) steps[k] = f2_of(0.0f, 0.0f);
        auto step = [&](int i) {
            f2 de[L::kCh], dx[L::kCh], bv[L::kSt];
            L::channels(de, &s.delta[i][p.local]);
            L::channels(dx, &s.dx[i][p.local]);
            L::states(bv, s.b + i * L::kStWidth + L::state_at((threadIdx.x & 31) % LS));
#pragma unroll
            for (int q = 0; q < L::kPairs; ++q) {
                const f2 decay = f2_decay(de[L::ci(q)], a2[q]);
                h[q] = f2_fma(dx[L::ci(q)], bv[L::si(q)], f2_mul(decay, h[q]));
            }
#pragma unroll
            for (int k = 0; k < L::kCh; ++k) steps[k] = f2_add(de[k], steps[k]);
        };
        if (rows == kTile) {
#pragma unroll 4
            for (int i = 0; i < kTile; ++i) step(i);
        } else {
            for (int i = 0; i < rows; ++i) step(i);
        }
#pragma unroll
        for (int k = 0; k < L::kCh; ++k) sum[k] = f2_add(sum[k], steps[k]);
    }
    store_states<LS, CPT>(a.tail + (int64_t)blockIdx.x * a.shape.channels * n, h, n, p.ch, p.count, p.n0);
    if ((threadIdx.x & 31) % LS == 0) {
        float* out = a.sum + (int64_t)blockIdx.x * a.shape.channels + p.ch;
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            float lo, hi;
            f2_split(sum[i / 2], lo, hi);
            if (i < p.count) out[i] = i & 1 ? hi : lo;
        }
    }
}

// 2. What each segment takes over, in the place of its tail.  Backward: from the
// last segment to the first.  32 states a CTA; its warps have a slice of the
// segments each, join it from nothing, learn through shared memory what the slices
// before come to, and go over theirs again.  76 segments of 1024 channels of 16
// states 10 us, 152 of 512 10 (one thread for a state: 12 us more over 187 of 512;
// a branch for far decays in place of halves: one trajectory of 2428 tokens, 432
// channels of 64 states, read 56.2 us against 54.9).
constexpr int kCarryWarps = 8, kAhead = 8;

struct Joined {      // carry <- 2^rate carry + own, or own alone
    float rate, own;
    bool open;
};

// Decays are kept as exponents until they meet a state, then in two halves: that of a
// state that grows may pass fp32's range, and a state of zero stays zero all the same
// (infinity times zero is no number).  2^254 takes every normal state past the range.
// Where the rate is no number, own is none either.
__device__ __forceinline__ float joined(const Joined& x, float carry) {
    const float half = exp2_of(fminf(x.rate, 254.0f) * 0.5f);
    return x.open ? fmaf(carry * half, half, x.own) : x.own;
}

__global__ void __launch_bounds__(32 * kCarryWarps) scan_carry_kernel(const __grid_constant__ Launch a, int backward) {
    __shared__ Joined slices[kCarryWarps][32];
    pdl_wait();
    pdl_trigger();
    const int n = a.shape.state_dim, lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int64_t states = (int64_t)a.shape.channels * n, i = (int64_t)blockIdx.x * 32 + lane;
    const bool on = i < states;
    const float a2 = on ? a.in.a[i] * kLog2e : 0.0f;
    const int64_t ch = i / n;
    const int each = (a.n_seg + kCarryWarps - 1) / kCarryWarps, lo = min(slice * each, a.n_seg), hi = min(lo + each, a.n_seg);
    // body(segment, what it makes of a carry), the loads of kAhead segments at once
    auto over = [&](auto&& body) {
        for (int from = lo; from < hi; from += kAhead) {
            float tail[kAhead], sum[kAhead];
            int kind[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int j = backward ? a.n_seg - 1 - (from + k) : from + k;
                kind[k] = kTailNone;
                if (on && from + k < hi) {
                    kind[k] = a.kind[j];
                    tail[k] = a.tail[j * states + i];
                    sum[k] = a.sum[(int64_t)j * a.shape.channels + ch];
                }
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (!on || from + k >= hi) break;
                const int j = backward ? a.n_seg - 1 - (from + k) : from + k;
                // selected, not multiplied: what an unused tail holds stays out
                Joined x = {0.0f, 0.0f, kind[k] == kTailJoin};
                if (kind[k] != kTailNone) x.own = tail[k];
                if (x.open) x.rate = a2 * sum[k];
                body(j, x);
            }
        }
    };
    Joined all = {0.0f, 0.0f, true};      // open: what came before the slice still counts
    over([&](int, const Joined& x) {
        all.own = joined(x, all.own);
        all.rate += x.rate;
        all.open = all.open && x.open;
    });
    slices[slice][lane] = all;
    __syncthreads();
    float carry = 0.0f;
    for (int k = 0; k < slice; ++k) carry = joined(slices[k][lane], carry);
    over([&](int j, const Joined& x) {
        a.tail[j * states + i] = carry;
        carry = joined(x, carry);
    });
}

// 3. The segments.  An update of a state is 4 fp32 operations, two states at a time,
// and an exp2 of its own, so the arithmetic bounds it before HBM does: 537 million
// updates are 57 us of fp32 and 54 of exp2 (34 a clock and SM, measured), 32768 tokens of
// 1024 channels of 16 states take 166, 65536 of 512, whose states are saved for the
// gradients, 187.  What is in between is issue, 61% busy (besides the states: softplus,
// gate and conversions of a token's channels, the sums over a channel's lanes), and
// L1 and shared memory, 72% busy.
template <typename T, int LS, int CPT>
__global__ void __launch_bounds__(kThreads, 4) scan_forward_kernel(const __grid_constant__ Launch a) {
    using L = Lay<LS, CPT>;
    using Ti = Tiling<T, L::CB, kTile>;
    extern __shared__ __align__(16) uint8_t dynamic[];
    auto& s = *reinterpret_cast<ForwardShared<T, LS, CPT>*>(dynamic);
    pdl_wait();
    const int tokens = (int)a.in.tokens, n = a.shape.state_dim;
    const int64_t row_states = (int64_t)a.shape.channels * n;
    const int s0 = (int)((int64_t)blockIdx.x * a.seg), s1 = (int)min((int64_t)s0 + a.seg, (int64_t)tokens);
    const Block b = block_at(a.shape, a.blocks, L::CB, blockIdx.y);
    const Place<LS, CPT> p(b);
    const bool mine = p.n0 < n;     // threads past the last state take no part in sums
    Rows<T, L::CB> x(a.in.x, a.in.x_stride, b, s0), dt(a.in.dt, a.in.dt_stride, b, s0), z(a.in.z, a.in.z_stride, b, s0);
    StatesHeld<T, LS, CPT> bs, cs;
    auto fetch = [&](int t0, int stage) {      // the tile after the ones asked for
        const int rows = min(kTile, s1 - t0);
        s.x[stage].ask(x, rows);
        s.dt.ask(dt, rows);
        bs.load(a.in.b, a.in.b_stride, b.group, n, t0, rows);
        cs.load(a.in.c, a.in.c_stride, b.group, n, t0, rows);
        x.move(1);
        dt.move(1);
    };
    s.x[0].clear();
    s.x[1].clear();
    s.dt.clear();
    if (s0 < s1) fetch(s0, 0);
    copies_commit();
    for (int i = threadIdx.x; i < kMaxSegment / 32; i += kThreads) s.mask[i] = 0;
    __syncthreads();
    if (threadIdx.x < 32) {
        const Range r = mark_starts(a.ends, a.episodes, tokens, s0, s1, s.mask);
        if (threadIdx.x == 0) s.range = r;
        if (blockIdx.y == 0) {
            const int bad = count_bad_ends(a.ends, a.episodes, tokens, blockIdx.x, gridDim.x);
            if (threadIdx.x == 0 && bad) atomicAdd(a.status + OFRL_STAT_BAD_INDEX, bad);
        }
    }
    f2 a2[L::kPairs], h[L::kPairs];
    load_decays<LS, CPT>(a2, a, p);
    float bias[Ti::V], skip[Ti::V];
    load_params<T, L::CB, kTile>(bias, a.in.dt_bias, b);
    load_params<T, L::CB, kTile>(skip, a.in.d, b);
    __syncthreads();
    const int end = s.range.end;
    int e = s.range.e0;
#pragma unroll
    for (int q = 0; q < L::kPairs; ++q) h[q] = f2_of(0.0f, 0.0f);
    if (s0 > 0 && s0 < end && !(s.mask[0] & 1))
        load_states<LS, CPT>(h, a.tail + (int64_t)blockIdx.x * row_states, n, p.ch, p.count, p.n0);

    auto leave = [&]() {     // the episode's last token is done
        if (a.final_state != nullptr && e < a.episodes)
            store_states<LS, CPT>(a.final_state + e * row_states, h, n, p.ch, p.count, p.n0);
    };
    int stage = 0;
    for (int t0 = s0; t0 < end; t0 += kTile, stage ^= 1) {
        const int rows = min(kTile, end - t0);
        copies_wait<0>();
        put_rows(s.delta, s.dx, s.x[stage], s.dt, bias, a.shape.softplus);
        bs.put(s.b);
        cs.put(s.c);
        __syncthreads();
        if (t0 + kTile < end) fetch(t0 + kTile, stage ^ 1);
        if (a.in.z != nullptr) {
            s.z.ask(z, rows);
            z.move(1);
        }
        copies_commit();
        const uint32_t starts = (s.mask[(t0 - s0) >> 5] >> ((t0 - s0) & 31)) & ((1u << kTile) - 1);
        // the state before token i, unless an episode begins there
        auto save = [&](int i) {
            if (a.saved != nullptr && !(starts >> i & 1))
                store_states<LS, CPT>(a.saved + (int64_t)((t0 + i) / kSave) * row_states, h, n, p.ch, p.count, p.n0);
        };
        // a token's part of sum_n C h, from this thread's states
        auto step = [&](int i, float (&y)[CPT]) {
            f2 de[L::kCh], dx[L::kCh], bv[L::kSt], cv[L::kSt];
            L::channels(de, &s.delta[i][p.local]);
            L::channels(dx, &s.dx[i][p.local]);
            const int at = i * L::kStWidth + L::state_at((threadIdx.x & 31) % LS);
            L::states(bv, s.b + at);
            L::states(cv, s.c + at);
            f2 acc[L::kCh];
#pragma unroll
            for (int q = 0; q < L::kPairs; ++q) {
                const f2 decay = f2_decay(de[L::ci(q)], a2[q]);
                h[q] = f2_fma(dx[L::ci(q)], bv[L::si(q)], f2_mul(decay, h[q]));
                acc[L::ci(q)] = L::si(q) == 0 ? f2_mul(cv[0], h[q]) : f2_fma(cv[L::si(q)], h[q], acc[L::ci(q)]);
            }
            if constexpr (CPT == 1) {
                y[0] = f2_sum(acc[0]);
            } else {
#pragma unroll
                for (int k = 0; k < L::kCh; ++k) f2_split(acc[k], y[2 * k], y[2 * k + 1]);
            }
            if (!mine)
#pragma unroll
                for (int k = 0; k < CPT; ++k) y[k] = 0.0f;
        };
        // the sums of tokens i .. take the place of their dx, which every lane has read
        auto put = [&](int i, float sum) {
            if (returns_channel<LS, CPT>()) s.dx[i][p.local + which_channel<LS, CPT>()] = sum;
        };
        if (starts == 0 && rows == kTile) {
            // four tokens between two barriers of the warp, so that their latencies overlap
            constexpr int kTogether = 4;
#pragma unroll 1
            for (int i = 0; i < kTile; i += kTogether) {
                if (i % kSave == 0) save(i);
                float y[kTogether][CPT], sum[kTogether];
#pragma unroll
                for (int k = 0; k < kTogether; ++k) step(i + k, y[k]);
#pragma unroll
                for (int k = 0; k < kTogether; ++k) sum[k] = sum_states<LS, CPT>(y[k]);
                __syncwarp();
#pragma unroll
                for (int k = 0; k < kTogether; ++k) put(i + k, sum[k]);
            }
        } else {
#pragma unroll 1
            for (int i = 0; i < rows; ++i) {
                if (i % kSave == 0) save(i);
                if (starts >> i & 1) {
                    if (t0 + i > s0) {
                        leave();
                        if (a.final_state != nullptr || a.init != nullptr)
                            e = next_episode(a.ends, e, a.episodes, tokens, t0 + i);
                    }
                    if (a.init != nullptr && e < a.episodes) {
                        load_states<LS, CPT>(h, a.init + e * row_states, n, p.ch, p.count, p.n0);
                    } else {
#pragma unroll
                        for (int q = 0; q < L::kPairs; ++q) h[q] = f2_of(0.0f, 0.0f);
                    }
                }
                float y[CPT];
                step(i, y);
                const float sum = sum_states<LS, CPT>(y);
                __syncwarp();
                put(i, sum);
            }
        }
        __syncthreads();
        copies_wait<0>();
        T* out = static_cast<T*>(a.out) + (int64_t)t0 * a.out_stride + b.ch0 + Ti::col();
#pragma unroll
        for (int j = 0; j < Ti::NV; ++j) {
            const int r = Ti::row(j);
            if (r >= rows || Ti::col() >= b.count) continue;
            const Vec<T, Ti::V> xv = s.x[stage].at(j), zv = s.z.at(j);
            float y[Ti::V];
#pragma unroll
            for (int i = 0; i < Ti::V; i += 2) {
                const float* q = &s.dx[r][Ti::col() + i];
                f2 v = f2_of(q[0], q[Ti::V > 1 ? 1 : 0]);
                if (a.in.d != nullptr) v = f2_fma(pair_at(skip, i), pair_of(xv, i), v);
                if (a.in.z != nullptr) v = f2_mul(v, silu(pair_of(zv, i)));
                set_pair(y, i, v);
            }
            store_vec<T, Ti::V>(out + r * a.out_stride, y);
        }
    }
    if (s.range.closed && end > s0) leave();

    // Episodes without tokens end as they began: every gridDim.x-th 32 of them.
    if (a.final_state != nullptr) {
        const int lane = threadIdx.x & 31;
        for (int64_t base = (int64_t)blockIdx.x * 32; base < a.episodes; base += (int64_t)gridDim.x * 32) {
            const int64_t at = base + lane;
            unsigned empty = __ballot_sync(0xffffffffu, at < a.episodes && episode_end(a.ends, (int)at, tokens) <=
                                                                             episode_start(a.ends, (int)at, tokens));
            for (; empty; empty &= empty - 1) {
                const int64_t ep = base + __ffs(empty) - 1;
                f2 v[L::kPairs];
#pragma unroll
                for (int q = 0; q < L::kPairs; ++q) v[q] = f2_of(0.0f, 0.0f);
                if (a.init != nullptr) load_states<LS, CPT>(v, a.init + ep * row_states, n, p.ch, p.count, p.n0);
                store_states<LS, CPT>(a.final_state + ep * row_states, v, n, p.ch, p.count, p.n0);
            }
        }
    }
}

template <typename T, int LS, int CPT>
cudaError_t go(const Launch& a, const Cut& c, cudaStream_t st) {
    static std::atomic<uint64_t> tail_done{0}, done{0};
    const dim3 grid((unsigned)c.n_seg, (unsigned)c.blocks);
    constexpr int tail_smem = (int)sizeof(TailShared<T, LS, CPT>), smem = (int)sizeof(ForwardShared<T, LS, CPT>);
    cudaError_t e = opt_in_once(scan_forward_kernel<T, LS, CPT>, smem, done);
    if (c.n_seg > 1) {
        if (e == cudaSuccess) e = opt_in_once(scan_tail_kernel<T, LS, CPT>, tail_smem, tail_done);
        if (e == cudaSuccess) e = launch_pdl(scan_tail_kernel<T, LS, CPT>, grid, dim3(kThreads), tail_smem, st, a);
        if (e == cudaSuccess) e = launch_carry(a, false, st);
    }
    if (e == cudaSuccess) e = launch_pdl(scan_forward_kernel<T, LS, CPT>, grid, dim3(kThreads), smem, st, a);
    return e;
}

template <typename T>
cudaError_t run(const Launch& a, const Cut& c, cudaStream_t st) {
    const bool wide = c.cpt > 1;
    switch (c.ls) {
        case 1: return go<T, 1, 1>(a, c, st);
        case 2: return wide ? go<T, 2, 2>(a, c, st) : go<T, 2, 1>(a, c, st);
        case 4: return wide ? go<T, 4, 4>(a, c, st) : go<T, 4, 1>(a, c, st);
        case 8: return wide ? go<T, 8, 4>(a, c, st) : go<T, 8, 1>(a, c, st);
        default: return wide ? go<T, 16, 4>(a, c, st) : go<T, 16, 1>(a, c, st);
    }
}

}  // namespace

cudaError_t launch_carry(const Launch& a, bool backward, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = opt_in_once(scan_carry_kernel, 0, done);
    const int64_t states = (int64_t)a.shape.channels * a.shape.state_dim;
    if (e == cudaSuccess)
        e = launch_pdl(scan_carry_kernel, dim3((unsigned)((states + 31) / 32)), dim3(32 * kCarryWarps), 0, st, a, (int)backward);
    return e;
}

cudaError_t launch_forward(const Launch& a, const Cut& c, cudaStream_t st) {
    return a.shape.dtype == OFRL_DTYPE_F32 ? run<float>(a, c, st) : run<__nv_bfloat16>(a, c, st);
}

}  // namespace scan
}  // namespace ofrl
