// Selective scan, gradients.
//
// With lam_t = dL/dh_t = dy_t C_t + a_{t+1} lam_{t+1}, dy = dout silu(z):
//   dx_t = delta_t sum_n lam_t B_t + D dy_t          dC_t = sum_d dy_t h_t
//   ddelta_t = x_t sum_n lam_t B_t + sum_n A lam_t p_t    dB_t = sum_d lam_t delta_t x_t
//   dA = sum_t delta_t lam_t p_t,  p_t = a_t h_{t-1},  h_t = p_t + delta_t B_t x_t.
// States come from the ones that the forward pass saved every kSave tokens: a tile
// is gone over forward, p kept in shared memory, then backward.  The sums over a
// token's channels (dB, dC) are made over the CTA's threads, then over the CTAs.
//
// 228 episodes of 64 to 512 tokens, 65536 in all, 512 channels of 16 states, bf16: tails
// 90 us, their join 7, the gradients 700, the joins of their parts 11.  The gradients'
// 15 fp32 operations and two exp2 for each state would be 230 us; a thread has 16
// states, 232 registers and 48 bytes of p and parts a state in shared memory, so an SM
// holds eight warps, which keep issue 47% and shared memory 56% busy.  (States saved
// every 16 tokens and two channels a thread: 74 us more.  The loops unrolled, or
// stores that loads may pass: no change.)

#include <cstddef>

#include "scan.cuh"

namespace ofrl {
namespace scan {
namespace {

constexpr int kBack = kSave;      // tokens of a tile: their p is in shared memory
// Tokens whose terms of dA are summed in registers, before they join the segment's sum
// in memory: one running sum over a segment of thousands rounds every term to its own size.
constexpr int kSum = 128;

template <int LS, int CPT>
struct GradShared {
    using L = Lay<LS, CPT>;
    static constexpr int kSlots = L::kPairs / 2 > 2 ? L::kPairs / 2 : 2;
    // of each token and channel: what the states need ...
    alignas(16) float delta[kBack][L::CB];
    alignas(16) float dx[kBack][L::CB];      // delta x
    alignas(16) float dy[kBack][L::CB];
    // ... and what its own gradients need besides
    alignas(16) float x[kBack][L::CB];
    alignas(16) float slope[kBack][L::CB];   // of delta by dt
    alignas(16) float gate[kBack][L::CB];    // dout silu'(z)
    alignas(16) float sum_b[kBack][L::CB];    // sum_n lam B
    alignas(16) float sum_a[kBack][L::CB];    // sum_n A2 lam p
    alignas(16) float y[kBack][L::CB];        // sum_n C h
    alignas(16) float b[kBack * L::kStWidth];
    alignas(16) float c[kBack * L::kStWidth];
    alignas(16) ulonglong2 p[kBack][kSlots][kThreads];      // then parts of dB and dC
    uint32_t mask[kMaxSegment / 32];
    Range range;
};

// dB and dC of a token are sums over the CTA's channels.  A thread's part, four
// floats of each, replaces the p it has just used; then every thread adds up
// what 128 / max(8, LS) threads with its states left for one (token, dB or dC),
// and lanes that share states add theirs.  (Summing over a warp's lanes by
// shuffles instead: 28 instructions more for each token.)
template <int LS, int SLOTS>
struct ChannelSums {
    static constexpr int kWidth = LS > 8 ? LS : 8;      // threads that read one sum's parts
    static constexpr int kAtOnce = kThreads / kWidth;   // sums of a round
    static constexpr int kRounds = 2 * kBack / kAtOnce;
    // put(row, half, first state, values) for each of the 2 count sums
    template <typename Put>
    __device__ static void run(const float4* parts, int count, const Put& put) {
        const int j = threadIdx.x % kWidth;
#pragma unroll
        for (int round = 0; round < kRounds; ++round) {
            const int rh = round * kAtOnce + (int)threadIdx.x / kWidth;
            float4 v = make_float4(0, 0, 0, 0);
#pragma unroll 8
            for (int k = j; k < kThreads; k += kWidth) {
                const float4 u = parts[((rh / 2) * SLOTS + rh % 2) * kThreads + k];
                v.x += u.x;
                v.y += u.y;
                v.z += u.z;
                v.w += u.w;
            }
#pragma unroll
            for (int o = LS; o < kWidth; o <<= 1) {
                v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
                v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
                v.z += __shfl_xor_sync(0xffffffffu, v.z, o);
                v.w += __shfl_xor_sync(0xffffffffu, v.w, o);
            }
            if (j < LS && rh / 2 < count) put(rh / 2, rh % 2, 4 * j, v);
        }
    }
};

// The row buffers of a call, tile by tile from the last: on their way in registers,
// then, as what their gradients are made of, in shared memory.
template <typename T, int CB, int ROWS, bool WITH_X>
struct TileHeld {
    using Ti = Tiling<T, CB, ROWS>;
    Rows<T, CB, ROWS> from_x, from_dt, from_z, from_g;
    RowsHeld<T, CB, ROWS> x, dt, z, g;
    __device__ TileHeld(const Launch& a, const Block& b, int t0)
        : from_x(a.in.x, a.in.x_stride, b, t0), from_dt(a.in.dt, a.in.dt_stride, b, t0),
          from_z(a.in.z, a.in.z_stride, b, t0), from_g(a.dout, a.dout_stride, b, t0) {}
    // the tile before the ones asked for
    __device__ void ask(const Launch& a, int rows) {
        if constexpr (WITH_X) x.ask(from_x, rows);
        dt.ask(from_dt, rows);
        if (a.in.z != nullptr) z.ask(from_z, rows);
        g.ask(from_g, rows);
        from_x.move(-1);
        from_dt.move(-1);
        from_z.move(-1);
        from_g.move(-1);
    }
    // delta and dy
    __device__ void put(float (*delta)[CB], float (*dy)[CB], const Launch& a, const float (&bias)[Ti::V]) const {
#pragma unroll
        for (int j = 0; j < Ti::NV; ++j) {
            const int r = Ti::row(j);
            if (r >= ROWS) continue;
            float d[Ti::V], gy[Ti::V];
#pragma unroll
            for (int i = 0; i < Ti::V; i += 2) {
                set_pair(d, i, delta_of(pair_of(dt.at(j), i), pair_at(bias, i), a.shape.softplus));
                f2 v = pair_of(g.at(j), i);
                if (a.in.z != nullptr) v = f2_mul(v, silu(pair_of(z.at(j), i)));
                set_pair(gy, i, v);
            }
            put_floats(&delta[r][Ti::col()], d);
            put_floats(&dy[r][Ti::col()], gy);
        }
    }
    template <typename S>
    __device__ void put_all(S& s, const Launch& a, const float (&bias)[Ti::V]) const {
#pragma unroll
        for (int j = 0; j < Ti::NV; ++j) {
            const int r = Ti::row(j);
            if (r >= ROWS) continue;
            float d[Ti::V], u[Ti::V], gy[Ti::V], xs[Ti::V], sl[Ti::V], gt[Ti::V];
#pragma unroll
            for (int i = 0; i < Ti::V; i += 2) {
                const f2 v = f2_add(pair_of(dt.at(j), i), pair_at(bias, i)), xv = pair_of(x.at(j), i);
                f2 slope = f2_both(1.0f), gv = pair_of(g.at(j), i);
                const f2 de = a.shape.softplus ? softplus_slope(v, slope) : v;
                if (a.in.z != nullptr) {
                    const f2 zv = pair_of(z.at(j), i), sg = sigmoid(zv);
                    set_pair(gt, i, f2_mul(gv, silu_slope(zv, sg)));
                    gv = f2_mul(gv, f2_mul(zv, sg));
                }
                set_pair(d, i, de);
                set_pair(u, i, f2_mul(de, xv));
                set_pair(gy, i, gv);
                set_pair(xs, i, xv);
                set_pair(sl, i, slope);
            }
            const int c = Ti::col();
            put_floats(&s.delta[r][c], d);
            put_floats(&s.dx[r][c], u);
            put_floats(&s.dy[r][c], gy);
            put_floats(&s.x[r][c], xs);
            put_floats(&s.slope[r][c], sl);
            if (a.in.z != nullptr) put_floats(&s.gate[r][c], gt);
        }
    }
};

// The adjoint a segment hands to the one before it.
template <typename T, int LS, int CPT>
__global__ void __launch_bounds__(kThreads) scan_grad_tail_kernel(const __grid_constant__ Launch a) {
    using L = Lay<LS, CPT>;
    using Ti = Tiling<T, L::CB, kTile>;
    __shared__ struct {
        alignas(16) float delta[kTile][L::CB];
        alignas(16) float dy[kTile][L::CB];
        alignas(16) float c[kTile * L::kStWidth];
        uint32_t mask[kMaxSegment / 32];
        Range range;
    } s;
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
    if ((s.mask[0] & 1) || s.range.end <= s0) {      // nothing goes to the segment before
        if (threadIdx.x == 0 && blockIdx.y == 0) a.kind[blockIdx.x] = kTailNone;
        return;
    }
    int end = s.range.end;
    bool own = s.range.closed;
    for (int w = 0; w <= (end - s0 - 1) >> 5; ++w)
        if (s.mask[w]) {
            end = s0 + w * 32 + __ffs(s.mask[w]) - 1;
            own = true;
            break;
        }
    if (threadIdx.x == 0 && blockIdx.y == 0) a.kind[blockIdx.x] = own ? kTailOwn : kTailJoin;

    const Block b = block_at(a.shape, a.blocks, L::CB, blockIdx.y);
    const Place<LS, CPT> p(b);
    f2 a2[L::kPairs], lam[L::kPairs], sum[L::kCh];
    load_decays<LS, CPT>(a2, a, p);
    float bias[Ti::V];
    load_params<T, L::CB, kTile>(bias, a.in.dt_bias, b);
#pragma unroll
    for (int i = 0; i < L::kCh; ++i) sum[i] = f2_of(0.0f, 0.0f);
#pragma unroll
    for (int q = 0; q < L::kPairs; ++q) lam[q] = f2_of(0.0f, 0.0f);
    if (own && a.d_final != nullptr && s.range.e0 < a.episodes)
        load_states<LS, CPT>(lam, a.d_final + (int64_t)s.range.e0 * a.shape.channels * n, n, p.ch, p.count, p.n0);
    const int last = s0 + (end - 1 - s0) / kTile * kTile;
    TileHeld<T, L::CB, kTile, false> rows_in(a, b, last);
    StatesHeld<T, LS, CPT> cs;
    auto fetch = [&](int t0) {
        const int rows = min(kTile, end - t0);
        rows_in.ask(a, rows);
        cs.load(a.in.c, a.in.c_stride, b.group, n, t0, rows);
    };
    fetch(last);
    for (int t0 = last; t0 >= s0; t0 -= kTile) {
        const int rows = min(kTile, end - t0);
        __syncthreads();      // the tile before is through
        rows_in.put(s.delta, s.dy, a, bias);
        cs.put(s.c);
        __syncthreads();
        if (t0 > s0) fetch(t0 - kTile);
        // the tile's deltas, from zero: one running sum over a segment rounds steps that hardly change
        // the same way for thousands of tokens (4096 of them 6e-5 off)
        f2 steps[L::kCh];
#pragma unroll
        for (int k = 0; k < L::kCh; ++k) steps[k] = f2_of(0.0f, 0.0f);
        auto step = [&](int i) {
            f2 de[L::kCh], gy[L::kCh], cv[L::kSt];
            L::channels(de, &s.delta[i][p.local]);
            L::channels(gy, &s.dy[i][p.local]);
            L::states(cv, s.c + i * L::kStWidth + L::state_at((threadIdx.x & 31) % LS));
#pragma unroll
            for (int q = 0; q < L::kPairs; ++q) {
                const f2 decay = f2_decay(de[L::ci(q)], a2[q]);
                lam[q] = f2_mul(decay, f2_fma(gy[L::ci(q)], cv[L::si(q)], lam[q]));
            }
#pragma unroll
            for (int k = 0; k < L::kCh; ++k) steps[k] = f2_add(de[k], steps[k]);
        };
        if (rows == kTile) {
#pragma unroll 4
            for (int i = kTile - 1; i >= 0; --i) step(i);
        } else {
            for (int i = rows - 1; i >= 0; --i) step(i);
        }
#pragma unroll
        for (int k = 0; k < L::kCh; ++k) sum[k] = f2_add(sum[k], steps[k]);
    }
    store_states<LS, CPT>(a.tail + (int64_t)blockIdx.x * a.shape.channels * n, lam, n, p.ch, p.count, p.n0);
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

// CTAs of an SM: what shared memory allows, and registers enough for them.
template <int LS, int CPT>
constexpr int grad_ctas() {
    constexpr int n = (227 * 1024) / ((int)sizeof(GradShared<LS, CPT>) + 1024);
    return n > 3 ? 3 : n;
}

template <typename T, int LS, int CPT>
__global__ void __launch_bounds__(kThreads, grad_ctas<LS, CPT>()) scan_grad_kernel(const __grid_constant__ Launch a) {
    using L = Lay<LS, CPT>;
    using Ti = Tiling<T, L::CB, kBack>;
    extern __shared__ __align__(16) uint8_t smem[];
    GradShared<LS, CPT>& s = *reinterpret_cast<GradShared<LS, CPT>*>(smem);
    pdl_wait();
    pdl_trigger();
    const int tokens = (int)a.in.tokens, n = a.shape.state_dim;
    const int64_t row_states = (int64_t)a.shape.channels * n;
    const int s0 = (int)((int64_t)blockIdx.x * a.seg), s1 = (int)min((int64_t)s0 + a.seg, (int64_t)tokens);
    for (int i = threadIdx.x; i < kMaxSegment / 32; i += kThreads) s.mask[i] = 0;
    __syncthreads();
    if (threadIdx.x < 32) {
        const Range r = mark_starts(a.ends, a.episodes, tokens, s0, s1, s.mask);
        if (threadIdx.x == 0) s.range = r;
    }
    const Block b = block_at(a.shape, a.blocks, L::CB, blockIdx.y);
    const Place<LS, CPT> p(b);
    const bool mine = p.n0 < n;
    const int parts = a.blocks / a.shape.groups;      // CTAs that share a group's dB and dC
    const int64_t dbc_stride = (int64_t)a.shape.groups * 2 * L::NP;
    float* dbc = a.dbc + (int64_t)(blockIdx.y % parts) * tokens * dbc_stride + b.group * 2 * L::NP;
    f2 a2[L::kPairs], da[L::kPairs], lam[L::kPairs], h[L::kPairs], next[L::kPairs];
    load_decays<LS, CPT>(a2, a, p);
    float bias[Ti::V], skip[Ti::V], dskip[Ti::V], dbias[Ti::V];
    load_params<T, L::CB, kBack>(bias, a.in.dt_bias, b);
    load_params<T, L::CB, kBack>(skip, a.in.d, b);
#pragma unroll
    for (int i = 0; i < Ti::V; ++i) dskip[i] = dbias[i] = 0.0f;
    const f2 zero = f2_of(0.0f, 0.0f);
#pragma unroll
    for (int q = 0; q < L::kPairs; ++q) da[q] = lam[q] = zero;
    __syncthreads();
    const int end = s.range.end;

    // the adjoint of an episode's last state, t its last token
    auto enter = [&](int t) {
#pragma unroll
        for (int q = 0; q < L::kPairs; ++q) lam[q] = zero;
        if (a.d_final == nullptr) return;
        const int e = find_episode(a.ends, 0, a.episodes, tokens, t);
        if (e < a.episodes) load_states<LS, CPT>(lam, a.d_final + e * row_states, n, p.ch, p.count, p.n0);
    };
    // the state before token t, which begins an episode
    auto begin = [&](int t) {
#pragma unroll
        for (int q = 0; q < L::kPairs; ++q) h[q] = zero;
        if (a.init == nullptr) return;
        const int e = find_episode(a.ends, 0, a.episodes, tokens, t);
        if (e < a.episodes) load_states<LS, CPT>(h, a.init + e * row_states, n, p.ch, p.count, p.n0);
    };
    float* const da_at = a.da + (int64_t)blockIdx.x * row_states;
    bool summed = false;
    auto sum_da = [&] {      // between tiles, where h is free
        if (summed) {
            load_states<LS, CPT>(h, da_at, n, p.ch, p.count, p.n0);
#pragma unroll
            for (int q = 0; q < L::kPairs; ++q) da[q] = f2_add(da[q], h[q]);
        }
        store_states<LS, CPT>(da_at, da, n, p.ch, p.count, p.n0);
#pragma unroll
        for (int q = 0; q < L::kPairs; ++q) da[q] = zero;
        summed = true;
    };
    const int last = s0 + (end - 1 - s0) / kBack * kBack;
    TileHeld<T, L::CB, kBack, true> rows_in(a, b, last);
    StatesHeld<T, LS, CPT, kBack> bs, cs;
    auto fetch = [&](int t0) {
        const int rows = min(kBack, end - t0);
        rows_in.ask(a, rows);
        bs.load(a.in.b, a.in.b_stride, b.group, n, t0, rows);
        cs.load(a.in.c, a.in.c_stride, b.group, n, t0, rows);
        // not written, and not used, where the tile begins an episode
        load_states<LS, CPT>(next, a.saved + (int64_t)(t0 / kBack) * row_states, n, p.ch, p.count, p.n0);
    };
    if (end > s0) {
        fetch(last);
        if (s.range.closed)
            enter(end - 1);
        else
            load_states<LS, CPT>(lam, a.tail + (int64_t)blockIdx.x * row_states, n, p.ch, p.count, p.n0);
    }
    const int at_state = L::state_at((threadIdx.x & 31) % LS);

    for (int t0 = last; t0 >= s0 && end > s0; t0 -= kBack) {
        const int rows = min(kBack, end - t0);
        rows_in.put_all(s, a, bias);      // the tile before is through
        bs.put(s.b);
        cs.put(s.c);
#pragma unroll
        for (int q = 0; q < L::kPairs; ++q) h[q] = next[q];
        __syncthreads();
        if (t0 > s0) fetch(t0 - kBack);
        const uint32_t starts = (s.mask[(t0 - s0) >> 5] >> ((t0 - s0) & 31)) & ((1u << kBack) - 1);
#pragma unroll 2
        for (int i = 0; i < rows; ++i) {
            if (starts >> i & 1) begin(t0 + i);
            f2 de[L::kCh], dx[L::kCh], bv[L::kSt], was[L::kPairs];
            L::channels(de, &s.delta[i][p.local]);
            L::channels(dx, &s.dx[i][p.local]);
            L::states(bv, s.b + i * L::kStWidth + at_state);
#pragma unroll
            for (int q = 0; q < L::kPairs; ++q) {
                was[q] = f2_mul(f2_decay(de[L::ci(q)], a2[q]), h[q]);
                h[q] = f2_fma(dx[L::ci(q)], bv[L::si(q)], was[q]);
            }
#pragma unroll
            for (int q = 0; q < L::kPairs; q += 2) s.p[i][q / 2][threadIdx.x] = make_ulonglong2(was[q], was[q + 1]);
        }
#pragma unroll 1
        for (int i = rows - 1; i >= 0; --i) {
            f2 de[L::kCh], dx[L::kCh], gy[L::kCh], bv[L::kSt], cv[L::kSt];
            L::channels(de, &s.delta[i][p.local]);
            L::channels(dx, &s.dx[i][p.local]);
            L::channels(gy, &s.dy[i][p.local]);
            L::states(bv, s.b + i * L::kStWidth + at_state);
            L::states(cv, s.c + i * L::kStWidth + at_state);
            f2 sb[L::kCh], sa[L::kCh], sy[L::kCh], db[L::kSt], dc[L::kSt];
#pragma unroll
            for (int q = 0; q < L::kPairs; ++q) {
                const int c = L::ci(q), k = L::si(q);
                const ulonglong2 two = s.p[i][q / 2][threadIdx.x];
                const f2 was = q & 1 ? two.y : two.x;
                const f2 now = f2_fma(dx[c], bv[k], was);
                const f2 l = f2_fma(gy[c], cv[k], lam[q]);
                const f2 w = f2_mul(l, was);
                dc[k] = c == 0 ? f2_mul(gy[c], now) : f2_fma(gy[c], now, dc[k]);
                db[k] = c == 0 ? f2_mul(l, dx[c]) : f2_fma(l, dx[c], db[k]);
                sb[c] = k == 0 ? f2_mul(l, bv[k]) : f2_fma(l, bv[k], sb[c]);
                sy[c] = k == 0 ? f2_mul(cv[k], now) : f2_fma(cv[k], now, sy[c]);
                sa[c] = k == 0 ? f2_mul(w, a2[q]) : f2_fma(w, a2[q], sa[c]);
                da[q] = f2_fma(w, de[c], da[q]);
                lam[q] = f2_mul(f2_decay(de[c], a2[q]), l);
            }
            float v[8], ch[3][CPT];
            if constexpr (L::kWide) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v[k] = f2_sum(db[k]);
                    v[4 + k] = f2_sum(dc[k]);
                }
#pragma unroll
                for (int k = 0; k < L::kCh; ++k) {
                    f2_split(sb[k], ch[0][2 * k], ch[0][2 * k + 1]);
                    f2_split(sa[k], ch[1][2 * k], ch[1][2 * k + 1]);
                    f2_split(sy[k], ch[2][2 * k], ch[2][2 * k + 1]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    f2_split(db[k], v[2 * k], v[2 * k + 1]);
                    f2_split(dc[k], v[4 + 2 * k], v[4 + 2 * k + 1]);
                }
                ch[0][0] = f2_sum(sb[0]);
                ch[1][0] = f2_sum(sa[0]);
                ch[2][0] = f2_sum(sy[0]);
            }
            if (n < L::NP)      // threads past the last state take no part in sums
#pragma unroll
                for (int k = 0; k < CPT; ++k)
                    if (!mine) ch[0][k] = ch[1][k] = ch[2][k] = 0.0f;
            float4* part = reinterpret_cast<float4*>(&s.p[i][0][threadIdx.x]);
            part[0] = make_float4(v[0], v[1], v[2], v[3]);
            part[kThreads] = make_float4(v[4], v[5], v[6], v[7]);
            const float to_b = sum_states<LS, CPT>(ch[0]), to_a = sum_states<LS, CPT>(ch[1]),
                        y = sum_states<LS, CPT>(ch[2]);
            if (returns_channel<LS, CPT>()) {
                const int at = p.local + which_channel<LS, CPT>();
                s.sum_b[i][at] = to_b;
                s.sum_a[i][at] = to_a;
                s.y[i][at] = y;
            }
            if (starts >> i & 1) {
                const int t = t0 + i;
                if (a.d_init != nullptr) {
                    const int e = find_episode(a.ends, 0, a.episodes, tokens, t);
                    if (e < a.episodes) store_states<LS, CPT>(a.d_init + e * row_states, lam, n, p.ch, p.count, p.n0);
                }
                if (t > s0) enter(t - 1);
            }
        }
        __syncthreads();
        // from shared memory to the gradients
        const int64_t ch = b.ch0 + Ti::col();
#pragma unroll
        for (int j = 0; j < Ti::NV; ++j) {
            const int r = Ti::row(j);
            if (r >= rows || Ti::col() >= b.count) continue;
            float out_x[Ti::V], out_dt[Ti::V], out_z[Ti::V];
            float d[Ti::V], to_b[Ti::V], gy[Ti::V], xs[Ti::V], sl[Ti::V], gt[Ti::V], to_a[Ti::V], y[Ti::V];
            load_vec<float, Ti::V>(d, &s.delta[r][Ti::col()]);
            load_vec<float, Ti::V>(to_b, &s.sum_b[r][Ti::col()]);
            load_vec<float, Ti::V>(gy, &s.dy[r][Ti::col()]);
            load_vec<float, Ti::V>(xs, &s.x[r][Ti::col()]);
            load_vec<float, Ti::V>(sl, &s.slope[r][Ti::col()]);
            load_vec<float, Ti::V>(to_a, &s.sum_a[r][Ti::col()]);
            if (a.in.z != nullptr) {
                load_vec<float, Ti::V>(gt, &s.gate[r][Ti::col()]);
                load_vec<float, Ti::V>(y, &s.y[r][Ti::col()]);
            }
#pragma unroll
            for (int k = 0; k < Ti::V; k += 2) {
                const f2 xv = pair_at(xs, k), gv = pair_at(gy, k), tb = pair_at(to_b, k), sk = pair_at(skip, k);
                f2 v = f2_mul(pair_at(d, k), tb);
                if (a.in.d != nullptr) v = f2_fma(sk, gv, v);
                set_pair(out_x, k, v);
                v = f2_mul(f2_fma(xv, tb, f2_mul(pair_at(to_a, k), f2_both(kLn2))), pair_at(sl, k));
                set_pair(out_dt, k, v);
                set_pair(dskip, k, f2_fma(gv, xv, pair_at(dskip, k)));
                set_pair(dbias, k, f2_add(v, pair_at(dbias, k)));
                if (a.in.z != nullptr) {
                    f2 yv = pair_at(y, k);
                    if (a.in.d != nullptr) yv = f2_fma(sk, xv, yv);
                    set_pair(out_z, k, f2_mul(pair_at(gt, k), yv));
                }
            }
            const int64_t t = t0 + r;
            store_vec<T, Ti::V>(static_cast<T*>(a.grads.dx) + t * a.grads.x_stride + ch, out_x);
            store_vec<T, Ti::V>(static_cast<T*>(a.grads.ddt) + t * a.grads.dt_stride + ch, out_dt);
            if (a.in.z != nullptr)
                store_vec<T, Ti::V>(static_cast<T*>(a.grads.dz) + t * a.grads.z_stride + ch, out_z);
        }
        ChannelSums<LS, GradShared<LS, CPT>::kSlots>::run(reinterpret_cast<const float4*>(s.p), rows, [&](int r, int half, int st, const float4& v) {
            const int64_t t = t0 + r;
            if (parts > 1) {
                *reinterpret_cast<float4*>(dbc + t * dbc_stride + half * L::NP + st) = v;
            } else if (st < n) {
                T* out = half ? static_cast<T*>(a.grads.dc) + t * a.grads.c_stride
                              : static_cast<T*>(a.grads.db) + t * a.grads.b_stride;
                out += b.group * n + st;
                out[0] = from_float<T>(v.x);
                out[1] = from_float<T>(v.y);
                out[2] = from_float<T>(v.z);
                out[3] = from_float<T>(v.w);
            }
        });
        if (t0 > s0 && (t0 - s0) % kSum == 0) sum_da();
        __syncthreads();
    }
    sum_da();
    // dD and ddt_bias over the threads of a column
    float(*red)[2][L::CB] = reinterpret_cast<float(*)[2][L::CB]>(&s.delta[0][0]);
    using S = GradShared<LS, CPT>;
    static_assert(sizeof(float) * Ti::kRowStep * 2 * L::CB <= offsetof(S, mask), "");
    put_floats(&red[threadIdx.x / Ti::kCols][0][Ti::col()], dskip);
    put_floats(&red[threadIdx.x / Ti::kCols][1][Ti::col()], dbias);
    __syncthreads();
    for (int c = threadIdx.x; c < b.count; c += kThreads) {
        float v = 0.0f, w = 0.0f;
        for (int k = 0; k < Ti::kRowStep; ++k) {
            v += red[k][0][c];
            w += red[k][1][c];
        }
        a.dd[(int64_t)blockIdx.x * a.shape.channels + b.ch0 + c] = v;
        a.dd[((int64_t)a.n_seg + blockIdx.x) * a.shape.channels + b.ch0 + c] = w;
    }

    // Episodes without tokens: the gradient passes through.
    if (a.d_init != nullptr) {
        const int lane = threadIdx.x & 31;
        for (int64_t base = (int64_t)blockIdx.x * 32; base < a.episodes; base += (int64_t)gridDim.x * 32) {
            const int64_t at = base + lane;
            unsigned empty = __ballot_sync(0xffffffffu, at < a.episodes && episode_end(a.ends, (int)at, tokens) <=
                                                                             episode_start(a.ends, (int)at, tokens));
            for (; empty; empty &= empty - 1) {
                const int64_t ep = base + __ffs(empty) - 1;
#pragma unroll
                for (int q = 0; q < L::kPairs; ++q) h[q] = zero;
                if (a.d_final != nullptr) load_states<LS, CPT>(h, a.d_final + ep * row_states, n, p.ch, p.count, p.n0);
                store_states<LS, CPT>(a.d_init + ep * row_states, h, n, p.ch, p.count, p.n0);
            }
        }
    }
}

// Joins the parts: dA, dD and ddt_bias over the segments, dB and dC over a
// group's CTAs.  CTAs [0, over): 32 outputs each, eight threads to an output;
// the rest: four outputs a thread.
constexpr int kJoinThreads = 256, kSlices = 8;

__device__ __forceinline__ float slice_sum(const float* p, int64_t stride, int parts, float (*red)[33]) {
    const int col = threadIdx.x % 32, slice = threadIdx.x / 32;
    float v = 0.0f;
    if (p != nullptr) {
#pragma unroll 8
        for (int j = slice; j < parts; j += kSlices) v += p[j * stride];
    }
    red[slice][col] = v;
    __syncthreads();
    float sum = 0.0f;
    if (slice == 0)
        for (int k = 0; k < kSlices; ++k) sum += red[k][col];
    return sum;
}

template <typename T>
__global__ void __launch_bounds__(kJoinThreads) scan_grad_join_kernel(const __grid_constant__ Launch a, int np, unsigned over) {
    __shared__ float red[kSlices][33];
    pdl_wait();
    const int n = a.shape.state_dim, d = a.shape.channels;
    if (blockIdx.x < over) {
        const int64_t states = (int64_t)d * n, i = (int64_t)blockIdx.x * 32 + threadIdx.x % 32;
        const float* p = nullptr;
        float* out = nullptr;
        int64_t stride = 0;
        if (i < states) {
            p = a.da + i;
            stride = states;
            out = a.grads.da + i;
        } else if (i < states + 2 * (int64_t)d) {
            const int64_t k = i - states;
            p = a.dd + (k < d ? k : (int64_t)a.n_seg * d + k - d);
            stride = d;
            out = k < d ? a.grads.dd : a.grads.ddt_bias;
            if (out != nullptr) out += k < d ? k : k - d;
        }
        const float v = slice_sum(p, stride, a.n_seg, red);
        if (threadIdx.x < 32 && out != nullptr) *out = v;
        return;
    }
    const int tokens = (int)a.in.tokens, live = episode_end(a.ends, a.episodes - 1, tokens);
    const int64_t per = (int64_t)a.shape.groups * 2 * np, total = (int64_t)live * per;
    const int parts = a.blocks / a.shape.groups;
    const int64_t i = (((int64_t)blockIdx.x - over) * kJoinThreads + threadIdx.x) * 4;
    if (i >= total) return;
    const int64_t t = i / per;
    const int rest = (int)(i - t * per), group = rest / (2 * np), k = rest % (2 * np), st = k % np;
    if (st >= n) return;
    float4 v = make_float4(0, 0, 0, 0);
#pragma unroll 8
    for (int j = 0; j < parts; ++j) {
        const float4 u = *reinterpret_cast<const float4*>(a.dbc + (int64_t)j * tokens * per + i);
        v.x += u.x;
        v.y += u.y;
        v.z += u.z;
        v.w += u.w;
    }
    T* out = k < np ? static_cast<T*>(a.grads.db) + t * a.grads.b_stride : static_cast<T*>(a.grads.dc) + t * a.grads.c_stride;
    out += group * n + st;
    out[0] = from_float<T>(v.x);
    out[1] = from_float<T>(v.y);
    out[2] = from_float<T>(v.z);
    out[3] = from_float<T>(v.w);
}

template <typename T>
cudaError_t join(const Launch& a, const Cut& c, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = opt_in_once(scan_grad_join_kernel<T>, 0, done);
    if (e != cudaSuccess) return e;
    const int np = 4 * c.ls;
    const int64_t outs = (int64_t)a.shape.channels * (a.shape.state_dim + 2), over = (outs + 31) / 32;
    int64_t more = 0;
    if (c.blocks > a.shape.groups)
        more = (a.in.tokens * a.shape.groups * 2 * np / 4 + kJoinThreads - 1) / kJoinThreads;
    if (over + more > INT32_MAX) return cudaErrorInvalidValue;
    return launch_ex(scan_grad_join_kernel<T>, dim3((unsigned)(over + more)), dim3(kJoinThreads), 0, st, 1, false, a, np,
                     (unsigned)over);
}

template <typename T, int LS, int CPT>
cudaError_t go(const Launch& a, const Cut& c, cudaStream_t st) {
    static std::atomic<uint64_t> tail_done{0}, done{0};
    const dim3 grid((unsigned)c.n_seg, (unsigned)c.blocks);
    const int smem = (int)sizeof(GradShared<LS, CPT>);
    cudaError_t e = opt_in_once(scan_grad_kernel<T, LS, CPT>, smem, done);
    if (c.n_seg > 1) {
        if (e == cudaSuccess) e = opt_in_once(scan_grad_tail_kernel<T, LS, CPT>, 0, tail_done);
        if (e == cudaSuccess) e = launch_pdl(scan_grad_tail_kernel<T, LS, CPT>, grid, dim3(kThreads), 0, st, a);
        if (e == cudaSuccess) e = launch_carry(a, true, st);
    }
    if (e == cudaSuccess) e = launch_pdl(scan_grad_kernel<T, LS, CPT>, grid, dim3(kThreads), smem, st, a);
    if (e == cudaSuccess) e = join<T>(a, c, st);
    return e;
}

template <typename T>
cudaError_t run(const Launch& a, const Cut& c, cudaStream_t st) {
    const bool wide = c.cpt == wide_of(c.ls);
    switch (c.ls) {
        case 1: return go<T, 1, 1>(a, c, st);
        case 2: return wide ? go<T, 2, 2>(a, c, st) : go<T, 2, 1>(a, c, st);
        case 4: return wide ? go<T, 4, 4>(a, c, st) : go<T, 4, 2>(a, c, st);
        case 8: return wide ? go<T, 8, 4>(a, c, st) : go<T, 8, 2>(a, c, st);
        default: return wide ? go<T, 16, 4>(a, c, st) : go<T, 16, 2>(a, c, st);
    }
}

}  // namespace

cudaError_t launch_backward(const Launch& a, const Cut& c, cudaStream_t st) {
    return a.shape.dtype == OFRL_DTYPE_F32 ? run<float>(a, c, st) : run<__nv_bfloat16>(a, c, st);
}

}  // namespace scan
}  // namespace ofrl
