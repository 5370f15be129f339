// Short causal convolution over packed episodes: forward, gradients, one token.
//
//   pre_t = bias + sum_{j < W} w_j x_{t-W+1+j},  out = act(pre)
//   dpre_t = dout_t act'(pre_t),  dx_t = sum_j w_{W-1-j} dpre_{t+j},
//   dw_j = sum_t dpre_t x_{t-W+1+j},  dbias = sum_t dpre_t
//
// A thread has a few neighbouring channels and goes down a run of tokens with
// the last W - 1 inputs in registers, so each input is read once but for the
// W - 1 tokens before a run (and, for gradients, after it).  Which tokens begin
// an episode is a bit mask in shared memory, made from the ends once a CTA.
// Bound by HBM in bytes; 65536 tokens of 1024 bf16 channels, four taps, silu:
// forward 51 us, 5.3 TB/s (the special functions' pipe 30% busy, issue 40%),
// gradients 88 us, 4.6 TB/s (issue 51%: two CTAs an SM, which their 126 registers
// allow, and instructions that wait for each other), their join 4 us; in fp32
// forward 93 us and gradients 140, 5.8 TB/s each.

#include <cstring>
#include <new>

#include "episodes.cuh"
#include "lanes.cuh"
#include "rows.cuh"

struct ofrl_conv {
    int device;
    int num_sms;
    ofrl_conv_shape shape;
    int64_t max_tokens;
    int32_t max_episodes;
    int32_t backward;
    void* base;          // the single cudaMalloc of the context
    int64_t bytes;
    int32_t* status;     // [OFRL_STAT_WORDS]
    float* parts;        // gradients: [CTAs over tokens][channels][width + 1]
};

namespace ofrl {
namespace {

constexpr int kThreads = 256;
// Channels of a thread: 16 bytes of them forward, four for gradients, whose
// taps, windows and sums would not stay in registers.
constexpr int vec_of(int elem, bool backward) { return elem == 4 || backward ? 4 : 8; }
constexpr int kMinRun = 8, kMaxRun = 256, kCtasPerSm = 2;
constexpr int kMaskWords = kThreads * kMaxRun / 32 + 4;

struct ConvLaunch {
    ofrl_conv_shape shape;
    ofrl_conv_tokens in;
    const int32_t* ends;
    int32_t episodes;
    const void* init;
    void* out;
    int64_t out_stride;
    void* final_state;
    const void* dout;
    int64_t dout_stride;
    const void* d_final;
    ofrl_conv_grads grads;
    float* d_init;
    float* parts;
    int32_t* status;
    int lanes;           // threads along a row, a power of two up to 32
    int run;             // tokens a thread goes down
};

struct ConvStepLaunch {
    ofrl_conv_shape shape;
    ofrl_conv_tokens in;
    const int32_t* slot_idx;
    int32_t slots;
    const void* state_in;
    void* state_out;
    void* out;
    int64_t out_stride;
    int32_t* status;
    int per_thread;      // tokens a thread takes
};

// How a call is cut: CTAs of (kThreads / lanes) runs by `lanes` vectors.
struct ConvCut {
    int lanes, run, cols;      // cols: CTAs along a row
    int64_t rows;              // CTAs over the tokens, at least 1
    int64_t fill;              // CTAs over the tokens that fill the GPU once
};
int64_t div_up(int64_t x, int64_t m) { return (x + m - 1) / m; }
ConvCut conv_cut(int channels, int vec, int64_t tokens, int num_sms) {
    ConvCut c;
    const int vecs = channels / vec;
    c.lanes = 1;
    while (c.lanes < 32 && c.lanes < vecs) c.lanes *= 2;
    c.cols = (int)div_up(vecs, c.lanes);
    const int64_t runs = kThreads / c.lanes;
    c.fill = div_up((int64_t)num_sms * kCtasPerSm, c.cols);
    const int64_t run = div_up(div_up(tokens, runs * c.fill), kMinRun) * kMinRun;
    c.run = (int)(run < kMinRun ? kMinRun : run > kMaxRun ? kMaxRun : run);
    c.rows = div_up(tokens, runs * c.run);
    if (c.rows < 1) c.rows = 1;
    return c;
}
// CTAs over the tokens of any call of at most max_tokens: at the longest run, or
// no more than fill the GPU.
int64_t conv_rows_most(int channels, int vec, int64_t max_tokens, int num_sms) {
    const ConvCut c = conv_cut(channels, vec, max_tokens, num_sms);
    const int64_t runs = kThreads / c.lanes, longest = div_up(max_tokens, runs * kMaxRun),
                  shortest = div_up(max_tokens, runs * kMinRun), few = c.fill < shortest ? c.fill : shortest;
    return longest > few ? longest : few > 1 ? few : 1;
}

__device__ __forceinline__ f2 act_of(f2 pre, int activation) { return activation == OFRL_ACT_SILU ? silu(pre) : pre; }
__device__ __forceinline__ f2 act_slope(f2 pre, int activation) {
    return activation == OFRL_ACT_SILU ? silu_slope(pre, sigmoid(pre)) : f2_both(1.0f);
}

// The first episode that ends after token t; one thread.
__device__ __forceinline__ int episode_at(const int32_t* ends, int episodes, int tokens, int t) {
    int lo = 0, hi = episodes;
    while (lo < hi) {
        const int mid = (int)(((int64_t)lo + hi) / 2);
        if (episode_end(ends, mid, tokens) > t)
            hi = mid;
        else
            lo = mid + 1;
    }
    return min(lo, episodes - 1);
}

// What a CTA knows of its tokens [s0, s1) and the W - 1 around them.
struct Marks {
    uint32_t mask[kMaskWords];
    int m0;              // the token of bit 0
    Range range;         // of [m0, ..)
    __device__ bool starts(int t) const { return mask[(t - m0) >> 5] >> ((t - m0) & 31) & 1; }
    // bit i: token t + i begins an episode, for 32 tokens from t >= m0 on
    __device__ uint32_t from(int t) const {
        const int o = t - m0;
        return __funnelshift_r(mask[o >> 5], mask[(o >> 5) + 1], o & 31);
    }
    // token t, below range.end, is its episode's last
    __device__ bool last(int t) const { return t + 1 < range.end ? starts(t + 1) : range.closed != 0; }
};

template <int W>
__device__ __forceinline__ void make_marks(Marks& m, const ConvLaunch& a, int s0, int64_t s1, bool count) {
    const int tokens = (int)a.in.tokens;
    for (int i = threadIdx.x; i < kMaskWords; i += kThreads) m.mask[i] = 0;
    __syncthreads();
    if (threadIdx.x < 32) {
        const int m0 = max(0, s0 - (W - 1)), m1 = (int)min(s1 + W, (int64_t)tokens);
        const Range r = mark_starts(a.ends, a.episodes, tokens, m0, max(m0, m1), m.mask);
        if (threadIdx.x == 0) {
            m.m0 = m0;
            m.range = r;
        }
        if (count) {
            const int bad = count_bad_ends(a.ends, a.episodes, tokens, blockIdx.x, gridDim.x);
            if (threadIdx.x == 0 && bad) atomicAdd(a.status + OFRL_STAT_BAD_INDEX, bad);
        }
    }
    __syncthreads();
}

// Inputs that a run carries along: win[i] stands W - 1 - i tokens back.
template <typename T, int V, int W>
struct Window {
    f2 win[W - 1][V / 2];
    __device__ void clear() {
#pragma unroll
        for (int i = 0; i < W - 1; ++i)
#pragma unroll
            for (int k = 0; k < V / 2; ++k) win[i][k] = f2_both(0.0f);
    }
    __device__ void push(const f2 (&x)[V / 2]) {
#pragma unroll
        for (int i = 0; i + 1 < W - 1; ++i)
#pragma unroll
            for (int k = 0; k < V / 2; ++k) win[i][k] = win[i + 1][k];
#pragma unroll
        for (int k = 0; k < V / 2; ++k) win[W - 2][k] = x[k];
    }
    // token t begins an episode
    __device__ void enter(const ConvLaunch& a, int t, int ch) {
        clear();
        if (a.init == nullptr) return;
        const int e = episode_at(a.ends, a.episodes, (int)a.in.tokens, t);
        const T* p = static_cast<const T*>(a.init) + ((int64_t)e * a.shape.channels + ch) * (W - 1);
#pragma unroll
        for (int k = 0; k < V / 2; ++k)
#pragma unroll
            for (int i = 0; i < W - 1; ++i)
                win[i][k] = f2_of(to_float(p[2 * k * (W - 1) + i]), to_float(p[(2 * k + 1) * (W - 1) + i]));
    }
    // token t ends an episode
    __device__ void leave(const ConvLaunch& a, int t, int ch) const {
        const int e = episode_at(a.ends, a.episodes, (int)a.in.tokens, t);
        T* p = static_cast<T*>(a.final_state) + ((int64_t)e * a.shape.channels + ch) * (W - 1);
#pragma unroll
        for (int k = 0; k < V / 2; ++k)
#pragma unroll
            for (int i = 0; i < W - 1; ++i) {
                p[2 * k * (W - 1) + i] = from_float<T>(f2_lo(win[i][k]));
                p[(2 * k + 1) * (W - 1) + i] = from_float<T>(f2_hi(win[i][k]));
            }
    }
};

template <int V, int W>
struct Taps {
    f2 w[W][V / 2], bias[V / 2];
    __device__ void load(const ConvLaunch& a, int ch) {
#pragma unroll
        for (int k = 0; k < V / 2; ++k) {
            const float* p = a.in.weight + (int64_t)(ch + 2 * k) * W;
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][k] = f2_of(p[j], p[W + j]);
            bias[k] = a.in.bias != nullptr ? f2_of(a.in.bias[ch + 2 * k], a.in.bias[ch + 2 * k + 1]) : f2_both(0.0f);
        }
    }
    template <typename T>
    __device__ f2 pre(const Window<T, V, W>& win, const f2 (&x)[V / 2], int k) const {
        f2 s = bias[k];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) s = f2_fma(w[j][k], win.win[j][k], s);
        return f2_fma(w[W - 1][k], x[k], s);
    }
};

// A run's inputs come through a ring in shared memory of which every thread has
// its own column: kRound tokens a group, kDepth groups on their way, no barrier.
// (The first inputs asked for after the marks, and several waves of CTAs: trained
// 196 us against 148.  Three groups 146.5, four 147.5, two 144; two of eight tokens
// 150; forward four channels a thread and three or four CTAs an SM 145.5 and 148.)
constexpr int kRound = 4, kDepth = 2;
template <typename T, int V, int N>
struct Ring {
    Vec<T, V> slot[N][kDepth][kRound][kThreads];
};

template <typename T, int W, int V>
__global__ void __launch_bounds__(kThreads, 2) conv_forward_kernel(const __grid_constant__ ConvLaunch a) {
    constexpr int P = V / 2, kBytes = V * (int)sizeof(T);
    extern __shared__ __align__(16) uint8_t dynamic[];
    Ring<T, V, 1>& ring = *reinterpret_cast<Ring<T, V, 1>*>(dynamic);
    __shared__ Marks m;
    pdl_wait();
    const int tokens = (int)a.in.tokens, d = a.shape.channels;
    const int runs = kThreads / a.lanes, lane = threadIdx.x % a.lanes, y = threadIdx.x / a.lanes;
    const int64_t from = (int64_t)blockIdx.x * runs * a.run;
    const int ch = ((int)blockIdx.y * a.lanes + lane) * V;
    const int64_t begin64 = from + (int64_t)y * a.run;
    // inputs are asked for before it is known which tokens episodes have
    const int bound = (int)min(begin64 + a.run, (int64_t)tokens), first = (int)min(max(begin64 - (W - 1), (int64_t)0), (int64_t)tokens);
    const T* in = static_cast<const T*>(a.in.x) + (int64_t)first * a.in.x_stride + ch;
    int left = bound - first, to = 0;      // tokens to be asked for yet, the next ones' group
    auto ask = [&]() {
#pragma unroll
        for (int i = 0; i < kRound; ++i) {
            if (ch < d && i < left) copy_async<kBytes>(&ring.slot[0][to][i][threadIdx.x], in);
            in += a.in.x_stride;
        }
        copies_commit();
        left -= kRound;
        to = to + 1 == kDepth ? 0 : to + 1;
    };
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) ask();
    make_marks<W>(m, a, (int)from, from + (int64_t)runs * a.run, blockIdx.y == 0);
    const int live = m.range.end, end = (int)min(begin64 + a.run, (int64_t)live), begin = (int)min(begin64, (int64_t)end);
    if (ch < d && begin < end) {
        T* out = static_cast<T*>(a.out) + (int64_t)first * a.out_stride + ch;
        Taps<V, W> taps;
        taps.load(a, ch);
        Window<T, V, W> win;
        win.clear();
        int group = 0;
        for (int t0 = first; t0 < end; t0 += kRound) {
            ask();
            copies_wait<kDepth - 1>();
            const uint32_t starts = m.from(t0);
            auto token = [&](int i, bool write) {
                const Vec<T, V> u = ring.slot[0][group][i][threadIdx.x];
                f2 x[P];
                Vec<T, V> o;
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    x[k] = vec_pair(u, k);
                    set_vec_pair(o, k, act_of(taps.pre(win, x, k), a.shape.activation));
                }
                if (write) *reinterpret_cast<Vec<T, V>*>(out) = o;
                out += a.out_stride;
                win.push(x);
            };
            // the usual round: whole, within the run and an episode
            if (t0 >= begin && t0 + kRound <= end && (starts & ((2u << kRound) - 1)) == 0 && t0 + kRound < live) {
#pragma unroll
                for (int i = 0; i < kRound; ++i) token(i, true);
            } else {
#pragma unroll 1
                for (int i = 0; i < kRound && t0 + i < end; ++i) {
                    const int t = t0 + i;
                    if (starts >> i & 1) win.enter(a, t, ch);
                    token(i, t >= begin);
                    if (a.final_state != nullptr && t >= begin && m.last(t)) win.leave(a, t, ch);
                }
            }
            group = group + 1 == kDepth ? 0 : group + 1;
        }
    }
    copies_wait<0>();
    // Episodes without tokens end as they began.
    if (a.final_state != nullptr) {
        const int ln = threadIdx.x & 31;
        const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
        const int ch0 = (int)blockIdx.y * a.lanes * V, width = min(a.lanes * V, d - ch0) * (W - 1);
        for (int64_t base = ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * 32; base < a.episodes;
             base += warps * 32) {
            const int64_t at = base + ln;
            unsigned empty = __ballot_sync(0xffffffffu, at < a.episodes && episode_end(a.ends, (int)at, tokens) <=
                                                                             episode_start(a.ends, (int)at, tokens));
            for (; empty; empty &= empty - 1) {
                const int64_t o = ((base + __ffs(empty) - 1) * d + ch0) * (W - 1);
                for (int i = ln; i < width; i += 32)
                    static_cast<T*>(a.final_state)[o + i] =
                        a.init != nullptr ? static_cast<const T*>(a.init)[o + i] : from_float<T>(0.0f);
            }
        }
    }
}

template <typename T, int W>
__global__ void __launch_bounds__(kThreads, 2) conv_grad_kernel(const __grid_constant__ ConvLaunch a) {
    constexpr int V = vec_of(sizeof(T), true), P = V / 2, kBytes = V * (int)sizeof(T);
    extern __shared__ __align__(16) uint8_t dynamic[];
    Ring<T, V, 2>& ring = *reinterpret_cast<Ring<T, V, 2>*>(dynamic);
    __shared__ Marks m;
    pdl_wait();
    pdl_trigger();
    const int tokens = (int)a.in.tokens, d = a.shape.channels;
    const int runs = kThreads / a.lanes, lane = threadIdx.x % a.lanes, y = threadIdx.x / a.lanes;
    const int64_t from = (int64_t)blockIdx.x * runs * a.run;
    const int ch = ((int)blockIdx.y * a.lanes + lane) * V;
    const int64_t begin64 = from + (int64_t)y * a.run;
    const int bound = (int)min(begin64 + a.run + W - 1, (int64_t)tokens), first = (int)min(max(begin64 - (W - 1), (int64_t)0), (int64_t)tokens);
    const T* in = static_cast<const T*>(a.in.x) + (int64_t)first * a.in.x_stride + ch;
    const T* go = static_cast<const T*>(a.dout) + (int64_t)first * a.dout_stride + ch;
    int left = bound - first, to = 0;      // tokens to be asked for yet, the next ones' group
    auto ask = [&]() {
#pragma unroll
        for (int i = 0; i < kRound; ++i) {
            if (ch < d && i < left) {
                copy_async<kBytes>(&ring.slot[0][to][i][threadIdx.x], in);
                copy_async<kBytes>(&ring.slot[1][to][i][threadIdx.x], go);
            }
            in += a.in.x_stride;
            go += a.dout_stride;
        }
        copies_commit();
        left -= kRound;
        to = to + 1 == kDepth ? 0 : to + 1;
    };
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) ask();
    make_marks<W>(m, a, (int)from, from + (int64_t)runs * a.run, false);
    const int live = m.range.end;
    const int end = (int)min(begin64 + a.run, (int64_t)live), begin = (int)min(begin64, (int64_t)end);
    f2 dw[W + 1][P];      // the taps, then the bias
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int k = 0; k < P; ++k) dw[j][k] = f2_both(0.0f);
    if (ch < d && begin < end) {
        const int stop = (int)min((int64_t)end + W - 1, (int64_t)live);      // dpre of the tokens after the run
        // dx of the token W - 1 before, which is complete: not dereferenced before the run begins
        T* out = static_cast<T*>(a.grads.dx) + (int64_t)(first - (W - 1)) * a.grads.x_stride + ch;
        Taps<V, W> taps;
        taps.load(a, ch);
        Window<T, V, W> win;
        win.clear();
        f2 pend[W - 1][P];      // dx of the W - 1 tokens before, so far
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int k = 0; k < P; ++k) pend[j][k] = f2_both(0.0f);
        int age = W;            // tokens since the episode began
        int group = 0;
        // W - 1 tokens more than the run: their gradients reach back into it
        for (int t0 = first; t0 < end + W - 1; t0 += kRound) {
            ask();
            copies_wait<kDepth - 1>();
            const uint32_t starts = m.from(t0);
            // a token's own dx is begun, those before it get their share (as far as `reach` back)
            auto token = [&](const f2 (&x)[P], int i, int reach, bool sums, f2 (&own)[P]) {
                const Vec<T, V> g = ring.slot[1][group][i][threadIdx.x];
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    const f2 dp = f2_mul(vec_pair(g, k), act_slope(taps.pre(win, x, k), a.shape.activation));
                    own[k] = f2_mul(taps.w[W - 1][k], dp);
#pragma unroll
                    for (int j = 1; j < W; ++j)
                        if (j <= reach) pend[W - 1 - j][k] = f2_fma(taps.w[W - 1 - j][k], dp, pend[W - 1 - j][k]);
                    if (sums) {
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) dw[j][k] = f2_fma(dp, win.win[j][k], dw[j][k]);
                        dw[W - 1][k] = f2_fma(dp, x[k], dw[W - 1][k]);
                        dw[W][k] = f2_add(dw[W][k], dp);
                    }
                }
            };
            auto take = [&](int i, f2 (&x)[P]) {
                const Vec<T, V> u = ring.slot[0][group][i][threadIdx.x];
#pragma unroll
                for (int k = 0; k < P; ++k) x[k] = vec_pair(u, k);
            };
            auto finish = [&](bool write, const f2 (&own)[P]) {      // the token W - 1 before is complete
                if (write) {
                    Vec<T, V> o;
#pragma unroll
                    for (int k = 0; k < P; ++k) set_vec_pair(o, k, pend[0][k]);
                    *reinterpret_cast<Vec<T, V>*>(out) = o;
                }
                out += a.grads.x_stride;
#pragma unroll
                for (int j = 0; j + 1 < W - 1; ++j)
#pragma unroll
                    for (int k = 0; k < P; ++k) pend[j][k] = pend[j + 1][k];
#pragma unroll
                for (int k = 0; k < P; ++k) pend[W - 2][k] = own[k];
            };
            // the usual round: whole, within the run and an episode, no gradient of a final state
            if (t0 >= begin + W - 1 && t0 + kRound <= end && (starts & ((1u << kRound) - 1)) == 0 && a.d_final == nullptr &&
                age >= W - 1) {
#pragma unroll
                for (int i = 0; i < kRound; ++i) {
                    f2 own[P], x[P];
                    take(i, x);
                    token(x, i, W - 1, true, own);
                    win.push(x);
                    finish(true, own);
                }
            } else {
#pragma unroll 1
                for (int i = 0; i < kRound; ++i) {
                    const int t = t0 + i, done = t - (W - 1);
                    f2 own[P], x[P];
#pragma unroll
                    for (int k = 0; k < P; ++k) own[k] = f2_both(0.0f);
                    if (t < stop) {
                        take(i, x);
                        if (starts >> i & 1) {
                            win.enter(a, t, ch);
                            age = 0;
                        }
                        if (t >= begin) {
                            token(x, i, age, t < end, own);
                            if (a.d_final != nullptr && t < end) {
                                int left = 0;      // tokens of the episode from t on, up to W - 1; 0: more
                                for (int j = 1; j < W && left == 0; ++j)
                                    if (t + j <= live && m.last(t + j - 1)) left = j;
                                if (left > 0) {
                                    const int e = episode_at(a.ends, a.episodes, tokens, t);
                                    const T* p = static_cast<const T*>(a.d_final) + ((int64_t)e * d + ch) * (W - 1) + W - 1 - left;
#pragma unroll
                                    for (int k = 0; k < P; ++k)
                                        own[k] = f2_add(own[k], f2_of(to_float(p[2 * k * (W - 1)]),
                                                                      to_float(p[(2 * k + 1) * (W - 1)])));
                                }
                            }
                        }
                        win.push(x);
                        age = min(age + 1, W);
                    }
                    finish(done >= begin && done < end, own);
                }
            }
            group = group + 1 == kDepth ? 0 : group + 1;
        }
    }
    copies_wait<0>();
    __syncthreads();
    float* red = reinterpret_cast<float*>(dynamic);
    static_assert(sizeof(Ring<T, V, 2>) >= sizeof(float) * kThreads * V * (W + 1), "");
    // over the CTA's runs
    const int row = a.lanes * V * (W + 1);
#pragma unroll
    for (int k = 0; k < P; ++k)
#pragma unroll
        for (int j = 0; j <= W; ++j) {
            float* p = red + y * row + (lane * V + 2 * k) * (W + 1) + j;
            p[0] = f2_lo(dw[j][k]);
            p[W + 1] = f2_hi(dw[j][k]);
        }
    __syncthreads();
    const int64_t first_out = (int64_t)blockIdx.y * row, all = (int64_t)d * (W + 1);
    for (int i = threadIdx.x; i < row && first_out + i < all; i += kThreads) {
        float v = 0.0f;
        for (int k = 0; k < runs; ++k) v += red[k * row + i];
        a.parts[blockIdx.x * all + first_out + i] = v;
    }
}

// dweight and dbias over the CTAs: 32 outputs a CTA, 32 threads to an output.
constexpr int kJoinThreads = 1024, kSlices = kJoinThreads / 32;

__global__ void __launch_bounds__(kJoinThreads) conv_join_kernel(const __grid_constant__ ConvLaunch a, int64_t rows) {
    __shared__ float red[kSlices][33];
    pdl_wait();
    if (a.d_init != nullptr) pdl_trigger();      // conv_init_grad_kernel is next
    const int w = a.shape.width;
    const int64_t all = (int64_t)a.shape.channels * (w + 1), i = (int64_t)blockIdx.x * 32 + threadIdx.x % 32;
    const int slice = threadIdx.x / 32;
    float v = 0.0f;
    if (i < all) {
#pragma unroll 8
        for (int64_t j = slice; j < rows; j += kSlices) v += a.parts[j * all + i];
    }
    red[slice][threadIdx.x % 32] = v;
    __syncthreads();
    if (slice > 0 || i >= all) return;
    v = 0.0f;
    for (int k = 0; k < kSlices; ++k) v += red[k][threadIdx.x];
    const int64_t ch = i / (w + 1);
    const int j = (int)(i - ch * (w + 1));
    if (j < w)
        a.grads.dweight[ch * w + j] = v;
    else if (a.grads.dbias != nullptr)
        a.grads.dbias[ch] = v;
}

// Gradient of the initial states: one thread for each episode and two channels,
// which goes over the first W - 1 tokens again.  Slot k stands W - 1 - k tokens
// before the episode: token i takes it with tap k - i.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads) conv_init_grad_kernel(const __grid_constant__ ConvLaunch a) {
    pdl_wait();
    const int tokens = (int)a.in.tokens, d = a.shape.channels;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x, e = i / (d / 2);
    const int ch = (int)(i - e * (d / 2)) * 2;
    if (e >= a.episodes) return;
    const int lo = episode_start(a.ends, (int)e, tokens), len = max(0, episode_end(a.ends, (int)e, tokens) - lo);
    Taps<2, W> taps;
    taps.load(a, ch);
    const int64_t at = (e * d + ch) * (W - 1);
    Window<T, 2, W> win;
    f2 g[W - 1];
    auto pair = [&](const void* p, int64_t o, int64_t apart) {
        const T* q = static_cast<const T*>(p) + o;
        return f2_of(to_float(q[0]), to_float(q[apart]));
    };
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        win.win[k][0] = a.init != nullptr ? pair(a.init, at + k, W - 1) : f2_both(0.0f);
        // a short episode's final state still holds initial inputs
        g[k] = a.d_final != nullptr && k >= len ? pair(a.d_final, at + k - len, W - 1) : f2_both(0.0f);
    }
#pragma unroll
    for (int t = 0; t < W - 1; ++t) {
        if (t >= len) break;
        const f2 x[1] = {pair(a.in.x, (int64_t)(lo + t) * a.in.x_stride + ch, 1)};
        const f2 dp = f2_mul(pair(a.dout, (int64_t)(lo + t) * a.dout_stride + ch, 1),
                             act_slope(taps.pre(win, x, 0), a.shape.activation));
#pragma unroll
        for (int k = t; k < W - 1; ++k) g[k] = f2_fma(taps.w[k - t][0], dp, g[k]);
        win.push(x);
    }
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        a.d_init[at + k] = f2_lo(g[k]);
        a.d_init[at + W - 1 + k] = f2_hi(g[k]);
    }
}

// One token of per_thread environments, eight channels a thread.  300 environments
// are a launch's latency; 16384 of 1024 channels, four taps, 133 us in bf16 and in fp32
// alike (2.0 and 4.1 TB/s), so not bytes bound them but a thread's loads, of weights one
// float at a time and of tokens one after the other.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(const __grid_constant__ ConvStepLaunch a) {
    constexpr int V = 16 / (int)sizeof(T), kVecs = 8 / V, S = W - 1;
    pdl_wait();
    const int d = a.shape.channels, cols = d / 8;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x, row = i / cols;
    const int ch = (int)(i - row * cols) * 8;
    const int64_t tok0 = row * a.per_thread, tok1 = min(tok0 + a.per_thread, a.in.tokens);
    if (tok0 >= tok1) return;
    float w[8][W], bias[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[k][j] = a.in.weight[(int64_t)(ch + k) * W + j];
        bias[k] = a.in.bias != nullptr ? a.in.bias[ch + k] : 0.0f;
    }
    for (int64_t tok = tok0; tok < tok1; ++tok) {
        const int32_t slot = a.slot_idx ? a.slot_idx[tok] : (int32_t)tok;
        T* out = static_cast<T*>(a.out) + tok * a.out_stride + ch;
        const bool ok = slot >= 0 && slot < a.slots;
        if (!ok && ch == 0) atomicAdd(a.status + OFRL_STAT_BAD_INDEX, 1);
        Vec<T, V> xv[kVecs], state[kVecs * S], o[kVecs];
        const T* x = static_cast<const T*>(a.in.x) + tok * a.in.x_stride + ch;
        const int64_t at = ((int64_t)(ok ? slot : 0) * d + ch) * S;
        if (ok) {
#pragma unroll
            for (int k = 0; k < kVecs * S; ++k)
                state[k] = *reinterpret_cast<const Vec<T, V>*>(static_cast<const T*>(a.state_in) + at + k * V);
#pragma unroll
            for (int k = 0; k < kVecs; ++k) xv[k] = *reinterpret_cast<const Vec<T, V>*>(x + k * V);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float s = bias[k];
#pragma unroll
                for (int j = 0; j < S; ++j) s = fmaf(w[k][j], to_float(state[(k * S + j) / V].v[(k * S + j) % V]), s);
                s = fmaf(w[k][S], to_float(xv[k / V].v[k % V]), s);
                o[k / V].v[k % V] = from_float<T>(a.shape.activation == OFRL_ACT_SILU ? s * sigmoid(s) : s);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
#pragma unroll
                for (int j = 0; j + 1 < S; ++j) state[(k * S + j) / V].v[(k * S + j) % V] =
                    state[(k * S + j + 1) / V].v[(k * S + j + 1) % V];
                state[(k * S + S - 1) / V].v[(k * S + S - 1) % V] = xv[k / V].v[k % V];
            }
#pragma unroll
            for (int k = 0; k < kVecs * S; ++k)
                *reinterpret_cast<Vec<T, V>*>(static_cast<T*>(a.state_out) + at + k * V) = state[k];
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k / V].v[k % V] = from_float<T>(0.0f);
        }
#pragma unroll
        for (int k = 0; k < kVecs; ++k) *reinterpret_cast<Vec<T, V>*>(out + k * V) = o[k];
    }
}

template <typename T, int W>
cudaError_t forward(const ConvLaunch& in, int num_sms, cudaStream_t st) {
    constexpr int V = vec_of(sizeof(T), false);
    static std::atomic<uint64_t> done{0};
    ConvLaunch a = in;
    const ConvCut c = conv_cut(a.shape.channels, V, a.in.tokens, num_sms);
    a.lanes = c.lanes;
    a.run = c.run;
    const cudaError_t e = opt_in_once(conv_forward_kernel<T, W, V>, (int)sizeof(Ring<T, V, 1>), done);
    if (e != cudaSuccess) return e;
    return launch_pdl(conv_forward_kernel<T, W, V>, dim3((unsigned)c.rows, (unsigned)c.cols), dim3(kThreads),
                      sizeof(Ring<T, V, 1>), st, a);
}

template <typename T, int W>
cudaError_t backward(const ConvLaunch& in, int num_sms, cudaStream_t st) {
    static std::atomic<uint64_t> done{0}, join_done{0}, init_done{0};
    ConvLaunch a = in;
    const ConvCut c = conv_cut(a.shape.channels, vec_of(sizeof(T), true), a.in.tokens, num_sms);
    a.lanes = c.lanes;
    a.run = c.run;
    const int64_t outs = (int64_t)a.shape.channels * (W + 1);
    using R = Ring<T, vec_of(sizeof(T), true), 2>;
    cudaError_t e = opt_in_once(conv_grad_kernel<T, W>, (int)sizeof(R), done);
    if (e == cudaSuccess) e = opt_in_once(conv_join_kernel, 0, join_done);
    if (e == cudaSuccess)
        e = launch_pdl(conv_grad_kernel<T, W>, dim3((unsigned)c.rows, (unsigned)c.cols), dim3(kThreads), sizeof(R), st, a);
    if (e == cudaSuccess)
        e = launch_pdl(conv_join_kernel, dim3((unsigned)((outs + 31) / 32)), dim3(kJoinThreads), 0, st, a, c.rows);
    if (e == cudaSuccess && a.d_init != nullptr) {
        const int64_t grid = ((int64_t)a.episodes * (a.shape.channels / 2) + kThreads - 1) / kThreads;
        if (grid > INT32_MAX) return cudaErrorInvalidValue;
        e = opt_in_once(conv_init_grad_kernel<T, W>, 0, init_done);
        if (e == cudaSuccess && grid > 0)
            e = launch_pdl(conv_init_grad_kernel<T, W>, dim3((unsigned)grid), dim3(kThreads), 0, st, a);
    }
    return e;
}

template <typename T, int W>
cudaError_t step(const ConvStepLaunch& in, int num_sms, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    ConvStepLaunch a = in;
    const int64_t cols = a.shape.channels / 8, full = (int64_t)num_sms * 4 * kThreads;
    // weights are loaded once a thread: more tokens a thread once the GPU is full
    a.per_thread = 1;
    while (a.per_thread < 8 && a.in.tokens * cols > full * 2 * a.per_thread) a.per_thread *= 2;
    const int64_t rows = (a.in.tokens + a.per_thread - 1) / a.per_thread, grid = (rows * cols + kThreads - 1) / kThreads;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    const cudaError_t e = opt_in_once(conv_step_kernel<T, W>, 0, done);
    return e != cudaSuccess ? e : launch_pdl(conv_step_kernel<T, W>, dim3((unsigned)grid), dim3(kThreads), 0, st, a);
}

// fn<T, W>(args...) for the shape's type and width.
#define OFRL_CONV_DISPATCH(shape, fn, ...)                                                                             \
    ((shape).dtype == OFRL_DTYPE_F32                                                                                   \
         ? ((shape).width == 2 ? fn<float, 2>(__VA_ARGS__)                                                             \
                               : (shape).width == 3 ? fn<float, 3>(__VA_ARGS__) : fn<float, 4>(__VA_ARGS__))           \
         : ((shape).width == 2 ? fn<__nv_bfloat16, 2>(__VA_ARGS__)                                                     \
                               : (shape).width == 3 ? fn<__nv_bfloat16, 3>(__VA_ARGS__)                                \
                                                    : fn<__nv_bfloat16, 4>(__VA_ARGS__)))

ofrl_status check_shape(const ofrl_conv_shape* s) {
    if (s == nullptr || s->channels < 1 || s->width < 1 || !dtype_ok(s->dtype) ||
        (s->activation != OFRL_ACT_NONE && s->activation != OFRL_ACT_SILU))
        return OFRL_EINVAL;
    if (s->channels > 65536 || s->channels % 8 != 0 || s->width < 2 || s->width > 4) return OFRL_EUNSUPPORTED;
    return OFRL_OK;
}

ofrl_status check_tokens(const ofrl_conv* ctx, const ofrl_conv_tokens* t) {
    if (t == nullptr || t->tokens < 0 || t->tokens > kMaxTokens) return OFRL_EINVAL;
    if (t->weight == nullptr || !aligned_to(t->weight, 4) || !aligned_to(t->bias, 4)) return OFRL_EINVAL;
    if (t->tokens > 0 && !rows_ok(t->x, t->x_stride, ctx->shape.channels, dtype_size(ctx->shape.dtype))) return OFRL_EINVAL;
    return OFRL_OK;
}

ofrl_status check_sequence(const ofrl_conv* ctx, const ofrl_conv_tokens* in, const int32_t* ends, int32_t episodes) {
    ofrl_status s = check_device(ctx);
    if (s == OFRL_OK) s = check_tokens(ctx, in);
    if (s != OFRL_OK) return s;
    if (episodes < 0 || (episodes > 0 && (ends == nullptr || !aligned_to(ends, 4)))) return OFRL_EINVAL;
    if (in->tokens > 0 && episodes == 0) return OFRL_EINVAL;
    if (in->tokens > ctx->max_tokens || episodes > ctx->max_episodes) return OFRL_EINVAL;
    return OFRL_OK;
}

int64_t conv_bytes(const ofrl_conv_shape& s, int64_t max_tokens, int num_sms, bool backward) {
    return 256 + (backward ? conv_rows_most(s.channels, vec_of(4, true), max_tokens, num_sms) * s.channels * (s.width + 1) * 4 : 0);
}

ConvLaunch base_launch(const ofrl_conv* ctx, const ofrl_conv_tokens* in, const int32_t* ends, int32_t episodes) {
    ConvLaunch a;
    std::memset(&a, 0, sizeof(a));
    a.shape = ctx->shape;
    a.in = *in;
    a.ends = ends;
    a.episodes = episodes;
    a.parts = ctx->parts;
    a.status = ctx->status;
    return a;
}

}  // namespace
}  // namespace ofrl

using namespace ofrl;

extern "C" {

int64_t ofrl_conv_workspace_bytes(const ofrl_conv_shape* shape, int64_t max_tokens, int32_t max_episodes,
                                  int32_t backward) {
    if (check_shape(shape) != OFRL_OK || !counts_ok(max_tokens, max_episodes) || (backward != 0 && backward != 1))
        return -1;
    int device = 0;
    const int sms = current_sms(&device);
    return conv_bytes(*shape, max_tokens, sms > 0 ? sms : 1, backward != 0);
}

ofrl_status ofrl_conv_create(const ofrl_conv_shape* shape, int64_t max_tokens, int32_t max_episodes, int32_t backward,
                             ofrl_conv** out) {
    if (out == nullptr) return OFRL_EINVAL;
    *out = nullptr;
    const ofrl_status s = check_shape(shape);
    if (s != OFRL_OK) return s;
    if (!counts_ok(max_tokens, max_episodes) || (backward != 0 && backward != 1)) return OFRL_EINVAL;
    ofrl_conv* ctx = new (std::nothrow) ofrl_conv;
    if (ctx == nullptr) return OFRL_ECUDA;
    std::memset(ctx, 0, sizeof(*ctx));
    ctx->num_sms = current_sms(&ctx->device);
    ctx->shape = *shape;
    ctx->max_tokens = max_tokens;
    ctx->max_episodes = max_episodes;
    ctx->backward = backward;
    if (ctx->num_sms > 0) ctx->bytes = conv_bytes(*shape, max_tokens, ctx->num_sms, backward != 0);
    if (ctx->num_sms == 0 || take_memory(&ctx->base, ctx->bytes) != cudaSuccess) {
        delete ctx;
        return OFRL_ECUDA;
    }
    ctx->status = static_cast<int32_t*>(ctx->base);
    ctx->parts = reinterpret_cast<float*>(static_cast<char*>(ctx->base) + 256);
    *out = ctx;
    return OFRL_OK;
}

ofrl_status ofrl_conv_destroy(ofrl_conv* ctx) { return release_memory(ctx); }

ofrl_status ofrl_conv_poll_status(ofrl_conv* ctx, void* stream, int32_t* words_out) {
    return poll_words(ctx, stream, words_out);
}

ofrl_status ofrl_conv_forward(ofrl_conv* ctx, const ofrl_conv_tokens* in, const int32_t* episode_ends,
                              int32_t num_episodes, const void* init_state, void* out, int64_t out_stride,
                              void* final_state, void* stream) {
    const ofrl_status s = check_sequence(ctx, in, episode_ends, num_episodes);
    if (s != OFRL_OK) return s;
    if (num_episodes == 0) return OFRL_OK;
    const int64_t e = dtype_size(ctx->shape.dtype);
    if (in->tokens > 0 && !rows_ok(out, out_stride, ctx->shape.channels, e)) return OFRL_EINVAL;
    if (!aligned_to(init_state, 16) || !aligned_to(final_state, 16)) return OFRL_EINVAL;
    const int64_t state = (int64_t)num_episodes * ctx->shape.channels * (ctx->shape.width - 1);
    if (overlap(init_state, state * e, final_state, state * e)) return OFRL_EINVAL;
    ConvLaunch a = base_launch(ctx, in, episode_ends, num_episodes);
    a.init = init_state;
    a.out = out;
    a.out_stride = out_stride;
    a.final_state = final_state;
    return cuda_status(OFRL_CONV_DISPATCH(ctx->shape, forward, a, ctx->num_sms, static_cast<cudaStream_t>(stream)));
}

ofrl_status ofrl_conv_backward(ofrl_conv* ctx, const ofrl_conv_tokens* in, const int32_t* episode_ends,
                               int32_t num_episodes, const void* init_state, const void* dout, int64_t dout_stride,
                               const void* d_final, const ofrl_conv_grads* grads, float* d_init, void* stream) {
    const ofrl_status s = check_sequence(ctx, in, episode_ends, num_episodes);
    if (s != OFRL_OK) return s;
    if (!ctx->backward || grads == nullptr || grads->dweight == nullptr) return OFRL_EINVAL;
    if (!aligned_to(grads->dweight, 4) || !aligned_to(grads->dbias, 4)) return OFRL_EINVAL;
    if (!aligned_to(init_state, 16) || !aligned_to(d_final, 16) || !aligned_to(d_init, 16)) return OFRL_EINVAL;
    const int64_t e = dtype_size(ctx->shape.dtype);
    if (in->tokens > 0 && (!rows_ok(dout, dout_stride, ctx->shape.channels, e) ||
                           !rows_ok(grads->dx, grads->x_stride, ctx->shape.channels, e)))
        return OFRL_EINVAL;
    const int64_t state = (int64_t)num_episodes * ctx->shape.channels * (ctx->shape.width - 1);
    if (overlap(init_state, state * e, d_init, state * 4) || overlap(d_final, state * e, d_init, state * 4))
        return OFRL_EINVAL;
    ConvLaunch a = base_launch(ctx, in, episode_ends, num_episodes);
    a.init = init_state;
    a.dout = dout;
    a.dout_stride = dout_stride;
    a.d_final = d_final;
    a.grads = *grads;
    a.d_init = d_init;
    return cuda_status(OFRL_CONV_DISPATCH(ctx->shape, backward, a, ctx->num_sms, static_cast<cudaStream_t>(stream)));
}

ofrl_status ofrl_conv_step(ofrl_conv* ctx, const ofrl_conv_tokens* in, const int32_t* slot_idx, int32_t slots,
                           const void* state_in, void* state_out, void* out, int64_t out_stride, void* stream) {
    ofrl_status s = check_device(ctx);
    if (s == OFRL_OK) s = check_tokens(ctx, in);
    if (s != OFRL_OK) return s;
    if (slots < 0 || !aligned_to(slot_idx, 4) || (slot_idx == nullptr && slots < in->tokens)) return OFRL_EINVAL;
    if (in->tokens == 0) return OFRL_OK;
    const int64_t e = dtype_size(ctx->shape.dtype);
    if (!rows_ok(out, out_stride, ctx->shape.channels, e)) return OFRL_EINVAL;
    if (!aligned_to(state_in, 16) || !aligned_to(state_out, 16)) return OFRL_EINVAL;
    if (slots > 0 && (!state_in || !state_out)) return OFRL_EINVAL;
    if (!same_or_apart(state_in, state_out, (int64_t)slots * ctx->shape.channels * (ctx->shape.width - 1) * e))
        return OFRL_EINVAL;
    ConvStepLaunch a;
    std::memset(&a, 0, sizeof(a));
    a.shape = ctx->shape;
    a.in = *in;
    a.slot_idx = slot_idx;
    a.slots = slots;
    a.state_in = state_in;
    a.state_out = state_out;
    a.out = out;
    a.out_stride = out_stride;
    a.status = ctx->status;
    return cuda_status(OFRL_CONV_DISPATCH(ctx->shape, step, a, ctx->num_sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
