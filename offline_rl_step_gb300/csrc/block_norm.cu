// Norms around a block: the gated norm after its memory and the norm of the
// residual stream before the next block; forward and gradients.
//
// With s = 1 / rms(u) over a group of W channels, e = dout (times the gate where
// it comes after the norm) and c = sum(e w u) / W:
//   out = w u s          du = s (e w - u s^2 c)          dw = sum over rows of e u s
// u is x, x silu(z), or h = residual + scale x.  Both sums of a row (u^2 and
// e w u) come from one read of it, which stays in registers until its outputs
// are written, so each tensor moves once.  Bound by HBM: 65536 rows of 1024 bf16
// channels, gated 62 us (6.5 TB/s), its gradients 116 (5.8); residual 84 (6.4), its
// gradients 132 (6.1); the join of the weights' gradients 5.
//
// A group of channels has up to 32 lanes of a warp, or a whole CTA.  Threads keep
// their columns over the rows they take, so a weight's gradient is a register until
// the end; then it is added over the CTA, and by a second launch over the CTAs, in a
// fixed order.

#include <cmath>
#include <cstring>
#include <new>

#include "lanes.cuh"
#include "rows.cuh"

struct ofrl_norm {
    int device;
    int num_sms;
    ofrl_norm_shape shape;
    int32_t backward;
    void* base;          // the single cudaMalloc of the context
    int64_t bytes;
    float* parts;        // gradients: [2][CTAs over rows][channels]
    int per_sm[2][2];    // CTAs an SM holds: [residual, gated][forward, backward]
};

namespace ofrl {
namespace {

constexpr int kWarpThreads = 128;        // of a CTA that has a warp or less for a group
constexpr int kMaxParts = 4096;          // CTAs over rows, at most
constexpr int kMostShared = 64 * 1024;   // weights and scales of 8192 channels

struct NormArgs {
    const void* x;
    const void* z;           // gated
    const void* residual;    // residual norm
    const float* scale;
    const float* weight;
    int64_t x_stride, z_stride, residual_stride;
    int64_t rows;
    float eps;
    int gate_first;
    int width;               // channels of a group
    int tg;                  // threads of a group
    void* out;
    int64_t out_stride;
    void* residual_out;
    int64_t residual_out_stride;
    const void* dout;
    int64_t dout_stride;
    const void* dres;        // gradient of residual_out, or null
    int64_t dres_stride;
    void* dx;
    int64_t dx_stride;
    void* dz;
    int64_t dz_stride;
    void* dresidual;
    int64_t dresidual_stride;
    float* parts;            // [2][gridDim.x][channels]
    int channels;
};

// What a launch's threads are to its rows: a group of channels is a warp's (or
// less) as long as a lane's elements, `most`, stay in registers, else a CTA's.
// (Eight elements a thread, more threads to a row: 5003 rows of 760 channels read
// 14.1 us against 8.9, 40000 rows of 1024 trained 166 against 124.)
struct NormCut {
    bool cta;
    int threads, tg, nv, groups_at_once;
};
NormCut norm_cut(int width, int elem, bool backward) {
    const int vec = 16 / elem, vecs = width / vec, most = (backward ? 16 : 32) / vec, most_cta = 16 / vec;
    NormCut c;
    c.cta = vecs > 32 * most;
    c.tg = c.cta ? 64 : 1;
    while (c.cta ? c.tg * most_cta < vecs : c.tg < 32 && c.tg < vecs) c.tg *= 2;
    c.threads = c.cta ? c.tg : kWarpThreads;
    const int nv = (vecs + c.tg - 1) / c.tg;
    c.nv = nv <= 1 ? 1 : nv <= 2 ? 2 : nv <= 4 ? 4 : 8;
    c.groups_at_once = c.threads / c.tg;
    return c;
}
// Floats of one weight row in shared memory, as the threads index it.
__host__ __device__ constexpr int weight_floats(int tg, int nv, int vec) { return tg * nv * vec; }

// Sums of N values over the group's threads, to all of them.
template <bool CTA, int N>
__device__ __forceinline__ void sum_group(float (&v)[N], int tg) {
    if constexpr (!CTA) {
        for (int o = tg >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    } else {
        __shared__ float p[16][N];
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) p[threadIdx.x >> 5][i] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 0.0f;
        for (int w = 0; w < tg / 32; ++w)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += p[w][i];
        __syncthreads();
    }
}

template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

// A thread's part of a row of S: NV times V elements, raw, zero past the group's
// width.  V is the vector of the row's narrower type, so fp32 beside bf16 takes two loads
// of 16 bytes for each.
template <typename S, int V, int NV>
struct Part {
    static constexpr int kPiece = V < 16 / (int)sizeof(S) ? V : 16 / (int)sizeof(S), kPieces = V / kPiece;
    Vec<S, kPiece> v[NV][kPieces];
    __device__ void load(const void* base, int64_t at, int lane, int tg, int width, bool on) {
        const S* p = static_cast<const S*>(base) + at;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (lane + j * tg) * V;
            if (on && c < width) {
#pragma unroll
                for (int i = 0; i < kPieces; ++i) v[j][i] = *reinterpret_cast<const Vec<S, kPiece>*>(p + c + i * kPiece);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) v[j][i / kPiece].v[i % kPiece] = from_float<S>(0.0f);
            }
        }
    }
    __device__ void store(void* base, int64_t at, int lane, int tg, int width) const {
        S* p = static_cast<S*>(base) + at;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (lane + j * tg) * V;
            if (c >= width) continue;
#pragma unroll
            for (int i = 0; i < kPieces; ++i) *reinterpret_cast<Vec<S, kPiece>*>(p + c + i * kPiece) = v[j][i];
        }
    }
    // elements 2 k and 2 k + 1 of vector j
    __device__ f2 pair(int j, int k) const { return vec_pair(v[j][2 * k / kPiece], k % (kPiece / 2)); }
    __device__ void set(int j, int k, f2 x) { set_vec_pair(v[j][2 * k / kPiece], k % (kPiece / 2), x); }
};

// The thread's place: which rows, which columns.
template <bool CTA>
struct Seat {
    int lane, at_once, seat;
    int64_t col0;            // the group's first channel
    __device__ explicit Seat(const NormArgs& a) {
        lane = CTA ? threadIdx.x : threadIdx.x % a.tg;
        at_once = CTA ? 1 : blockDim.x / a.tg;
        seat = CTA ? 0 : threadIdx.x / a.tg;
        col0 = (int64_t)blockIdx.y * a.width;
    }
};

__device__ __forceinline__ float rstd_of(float squares, const NormArgs& a) {
    return rsqrtf(squares / (float)a.width + a.eps);
}

// The group's weights (and scales) in shared memory, zero past its width: four
// floats of each lane side by side, so that lanes read without conflicts.
template <int V, int NV>
__device__ __forceinline__ void stage_weights(float* dst, const float* src, const NormArgs& a) {
    const int n = weight_floats(a.tg, NV, V) / 4;      // a.tg is a power of two
    const int log_tg = 31 - __clz(a.tg);
    const float4* from = reinterpret_cast<const float4*>(src + (int64_t)blockIdx.y * a.width);
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int vec = i / (V / 4), piece = i % (V / 4), lane = vec & (a.tg - 1), j = vec >> log_tg;
        reinterpret_cast<float4*>(dst)[(((j * (V / 4) + piece) << log_tg) + lane)] =
            4 * i < a.width ? from[i] : make_float4(0, 0, 0, 0);
    }
}
template <int V>
struct Weights {
    const ulonglong2* p;
    int tg;
    __device__ Weights(const float* base, int lane, int tg_) : p(reinterpret_cast<const ulonglong2*>(base) + lane), tg(tg_) {}
    __device__ void load(f2 (&w)[V / 2], int j) const {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const ulonglong2 u = p[(j * (V / 4) + i) * tg];
            w[2 * i] = u.x;
            w[2 * i + 1] = u.y;
        }
    }
};

// Rows go by, row(i, on) each.  Few elements a thread: the next row's loads are in
// flight meanwhile (fetch); more of them: it is on its way to L2 (ask).  The first
// row is asked for before the weights are staged.
template <int ELEMENTS, bool CTA, typename Ask, typename Fetch, typename Stage, typename Row>
__device__ __forceinline__ void for_rows(const NormArgs& a, const Seat<CTA>& s, const Ask& ask, const Fetch& fetch,
                                         const Stage& stage, const Row& row) {
    constexpr bool kAhead = ELEMENTS <= 8;
    const int64_t step = (int64_t)gridDim.x * s.at_once;
    int64_t row0 = (int64_t)blockIdx.x * s.at_once;
    if (kAhead)
        fetch(row0 + s.seat, row0 + s.seat < a.rows);
    else if (s.lane == 0 && row0 + s.seat < a.rows)
        ask(row0 + s.seat);
    stage();
    __syncthreads();
    for (; row0 < a.rows; row0 += step) {
        const int64_t i = row0 + s.seat, after = i + step;
        if (!kAhead) {
            fetch(i, i < a.rows);
            if (s.lane == 0 && after < a.rows) ask(after);
        }
        row(i, i < a.rows, [&]() {
            if (kAhead) fetch(after, after < a.rows);
        });
    }
}
// A row's part of one tensor, to L2.
template <typename S>
__device__ __forceinline__ void ask_row(const NormArgs& a, const void* base, int64_t at) {
    prefetch_l2(static_cast<const S*>(base) + at, (uint32_t)(a.width * sizeof(S)));
}

template <typename T, int NV, bool CTA>
__global__ void __launch_bounds__(CTA ? 512 : kWarpThreads) gated_norm_kernel(const __grid_constant__ NormArgs a) {
    constexpr int V = kVec<T>;
    extern __shared__ __align__(16) float dynamic[];
    pdl_wait();
    const Seat<CTA> s(a);
    auto stage = [&]() { stage_weights<V, NV>(dynamic, a.weight, a); };
    const Weights<V> w(dynamic, s.lane, a.tg);
    Part<T, V, NV> next_x, next_z;
    auto fetch = [&](int64_t row, bool on) {
        next_x.load(a.x, row * a.x_stride + s.col0, s.lane, a.tg, a.width, on);
        next_z.load(a.z, row * a.z_stride + s.col0, s.lane, a.tg, a.width, on);
    };
    auto ask = [&](int64_t row) {
        ask_row<T>(a, a.x, row * a.x_stride + s.col0);
        ask_row<T>(a, a.z, row * a.z_stride + s.col0);
    };
    for_rows<NV * V>(a, s, ask, fetch, stage, [&](int64_t row, bool on, auto loaded) {
        Part<T, V, NV> x = next_x, z = next_z;
        loaded();
        f2 sq = f2_both(0.0f);
        // the gate first: u = x silu(z) is needed twice and rounded nowhere
        f2 u[NV][V / 2];
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < V / 2; ++k) {
                u[j][k] = x.pair(j, k);
                if (a.gate_first) u[j][k] = f2_mul(u[j][k], silu(z.pair(j, k)));
                sq = f2_fma(u[j][k], u[j][k], sq);
            }
        float sum[1] = {f2_sum(sq)};
        sum_group<CTA>(sum, a.tg);
        const f2 r = f2_both(rstd_of(sum[0], a));
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            f2 wv[V / 2];
            w.load(wv, j);
#pragma unroll
            for (int k = 0; k < V / 2; ++k) {
                f2 g = f2_mul(r, wv[k]);
                if (!a.gate_first) g = f2_mul(g, silu(z.pair(j, k)));
                x.set(j, k, f2_mul(u[j][k], g));
            }
        }
        if (on) x.store(a.out, row * a.out_stride + s.col0, s.lane, a.tg, a.width);
    });
}

// T: x and out, R: the residual.
template <typename T, typename R, int NV, bool CTA>
__global__ void __launch_bounds__(CTA ? 512 : kWarpThreads) residual_norm_kernel(const __grid_constant__ NormArgs a) {
    constexpr int V = kVec<T>;
    extern __shared__ __align__(16) float dynamic[];
    pdl_wait();
    const Seat<CTA> s(a);
    float* scales = dynamic + weight_floats(a.tg, NV, V);
    auto stage = [&]() {
        stage_weights<V, NV>(dynamic, a.weight, a);
        if (a.scale != nullptr) stage_weights<V, NV>(scales, a.scale, a);
    };
    const Weights<V> w(dynamic, s.lane, a.tg), scale(scales, s.lane, a.tg);
    Part<T, V, NV> next_x;
    Part<R, V, NV> next_h;
    auto fetch = [&](int64_t row, bool on) {
        next_x.load(a.x, row * a.x_stride + s.col0, s.lane, a.tg, a.width, on);
        next_h.load(a.residual, row * a.residual_stride + s.col0, s.lane, a.tg, a.width, on);
    };
    auto ask = [&](int64_t row) {
        ask_row<T>(a, a.x, row * a.x_stride + s.col0);
        ask_row<R>(a, a.residual, row * a.residual_stride + s.col0);
    };
    for_rows<NV * V>(a, s, ask, fetch, stage, [&](int64_t row, bool on, auto loaded) {
        Part<T, V, NV> x = next_x;
        Part<R, V, NV> res = next_h;
        loaded();
        f2 h[NV][V / 2], sq = f2_both(0.0f);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            f2 sc[V / 2];
            if (a.scale != nullptr) scale.load(sc, j);
#pragma unroll
            for (int k = 0; k < V / 2; ++k) {
                h[j][k] = a.scale != nullptr ? f2_fma(sc[k], x.pair(j, k), res.pair(j, k))
                                             : f2_add(x.pair(j, k), res.pair(j, k));
                sq = f2_fma(h[j][k], h[j][k], sq);
                res.set(j, k, h[j][k]);
            }
        }
        if (on) res.store(a.residual_out, row * a.residual_out_stride + s.col0, s.lane, a.tg, a.width);
        float sum[1] = {f2_sum(sq)};
        sum_group<CTA>(sum, a.tg);
        const f2 r = f2_both(rstd_of(sum[0], a));
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            f2 wv[V / 2];
            w.load(wv, j);
#pragma unroll
            for (int k = 0; k < V / 2; ++k) x.set(j, k, f2_mul(f2_mul(h[j][k], r), wv[k]));
        }
        if (on) x.store(a.out, row * a.out_stride + s.col0, s.lane, a.tg, a.width);
    });
}

// A thread's sums over its rows of one weight's gradient.
template <int V, int NV>
struct ColumnSums {
    f2 v[NV][V / 2];
    __device__ ColumnSums() {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < V / 2; ++k) v[j][k] = f2_both(0.0f);
    }
    // over the CTA's seats, to the CTA's place in parts; red holds a row a seat
    template <bool CTA>
    __device__ void put(const NormArgs& a, const Seat<CTA>& s, int which, float* red) const {
        float* out = a.parts + ((int64_t)which * gridDim.x + blockIdx.x) * a.channels + s.col0;
        const int row = weight_floats(a.tg, NV, V);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < V / 2; ++k)
                *reinterpret_cast<f2*>(red + s.seat * row + (s.lane + j * a.tg) * V + 2 * k) = v[j][k];
        __syncthreads();
        for (int c = threadIdx.x; c < a.width; c += blockDim.x) {
            float x = 0.0f;
            for (int i = 0; i < s.at_once; ++i) x += red[i * row + c];
            out[c] = x;
        }
    }
};

template <typename T, int NV, bool CTA>
__global__ void __launch_bounds__(CTA ? 512 : kWarpThreads) gated_norm_grad_kernel(const __grid_constant__ NormArgs a) {
    constexpr int V = kVec<T>;
    extern __shared__ __align__(16) float dynamic[];
    pdl_wait();
    pdl_trigger();
    const Seat<CTA> s(a);
    auto stage = [&]() { stage_weights<V, NV>(dynamic, a.weight, a); };
    const Weights<V> w(dynamic, s.lane, a.tg);
    ColumnSums<V, NV> dw;
    Part<T, V, NV> next_x, next_z, next_g;
    auto fetch = [&](int64_t row, bool on) {
        next_x.load(a.x, row * a.x_stride + s.col0, s.lane, a.tg, a.width, on);
        next_z.load(a.z, row * a.z_stride + s.col0, s.lane, a.tg, a.width, on);
        next_g.load(a.dout, row * a.dout_stride + s.col0, s.lane, a.tg, a.width, on);
    };
    auto ask = [&](int64_t row) {
        ask_row<T>(a, a.x, row * a.x_stride + s.col0);
        ask_row<T>(a, a.z, row * a.z_stride + s.col0);
        ask_row<T>(a, a.dout, row * a.dout_stride + s.col0);
    };
    for_rows<NV * V>(a, s, ask, fetch, stage, [&](int64_t row, bool on, auto loaded) {
        Part<T, V, NV> x = next_x, z = next_z, g = next_g;
        loaded();
        f2 sq = f2_both(0.0f), ip = f2_both(0.0f), sg[NV][V / 2];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            f2 wv[V / 2];
            w.load(wv, j);
#pragma unroll
            for (int k = 0; k < V / 2; ++k) {
                const f2 zv = z.pair(j, k);
                sg[j][k] = sigmoid(zv);
                const f2 gate = f2_mul(zv, sg[j][k]);
                f2 u = x.pair(j, k), e = g.pair(j, k);
                if (a.gate_first)
                    u = f2_mul(u, gate);
                else
                    e = f2_mul(e, gate);
                sq = f2_fma(u, u, sq);
                ip = f2_fma(f2_mul(e, wv[k]), u, ip);
            }
        }
        float sum[2] = {f2_sum(sq), f2_sum(ip)};
        sum_group<CTA>(sum, a.tg);
        const float rs = rstd_of(sum[0], a);
        const f2 r = f2_both(rs), back = f2_both(-rs * rs * sum[1] / (float)a.width);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            f2 wv[V / 2];
            w.load(wv, j);
#pragma unroll
            for (int k = 0; k < V / 2; ++k) {
                const f2 zv = z.pair(j, k), gate = f2_mul(zv, sg[j][k]), xv = x.pair(j, k), gv = g.pair(j, k);
                const f2 u = a.gate_first ? f2_mul(xv, gate) : xv, e = a.gate_first ? gv : f2_mul(gv, gate);
                const f2 unit = f2_mul(u, r), du = f2_mul(r, f2_fma(e, wv[k], f2_mul(u, back)));
                dw.v[j][k] = f2_fma(e, unit, dw.v[j][k]);
                const f2 dgate = a.gate_first ? f2_mul(du, xv) : f2_mul(f2_mul(gv, unit), wv[k]);
                x.set(j, k, a.gate_first ? f2_mul(du, gate) : du);
                z.set(j, k, f2_mul(dgate, silu_slope(zv, sg[j][k])));
            }
        }
        if (on) {
            x.store(a.dx, row * a.dx_stride + s.col0, s.lane, a.tg, a.width);
            z.store(a.dz, row * a.dz_stride + s.col0, s.lane, a.tg, a.width);
        }
    });
    dw.put(a, s, 0, dynamic);
}

template <typename T, typename R, int NV, bool CTA>
__global__ void __launch_bounds__(CTA ? 512 : kWarpThreads) residual_norm_grad_kernel(const __grid_constant__ NormArgs a) {
    constexpr int V = kVec<T>;
    extern __shared__ __align__(16) float dynamic[];
    pdl_wait();
    pdl_trigger();
    const Seat<CTA> s(a);
    float* scales = dynamic + weight_floats(a.tg, NV, V);
    auto stage = [&]() {
        stage_weights<V, NV>(dynamic, a.weight, a);
        if (a.scale != nullptr) stage_weights<V, NV>(scales, a.scale, a);
    };
    const Weights<V> w(dynamic, s.lane, a.tg), scale(scales, s.lane, a.tg);
    ColumnSums<V, NV> dw, ds;
    Part<T, V, NV> next_x, next_g;
    Part<R, V, NV> next_h, next_d;
    auto fetch = [&](int64_t row, bool on) {
        next_x.load(a.x, row * a.x_stride + s.col0, s.lane, a.tg, a.width, on);
        next_h.load(a.residual, row * a.residual_stride + s.col0, s.lane, a.tg, a.width, on);
        next_g.load(a.dout, row * a.dout_stride + s.col0, s.lane, a.tg, a.width, on);
        next_d.load(a.dres, row * a.dres_stride + s.col0, s.lane, a.tg, a.width, on && a.dres != nullptr);
    };
    auto ask = [&](int64_t row) {
        ask_row<T>(a, a.x, row * a.x_stride + s.col0);
        ask_row<R>(a, a.residual, row * a.residual_stride + s.col0);
        ask_row<T>(a, a.dout, row * a.dout_stride + s.col0);
        if (a.dres != nullptr) ask_row<R>(a, a.dres, row * a.dres_stride + s.col0);
    };
    for_rows<NV * V>(a, s, ask, fetch, stage, [&](int64_t row, bool on, auto loaded) {
        Part<T, V, NV> x = next_x, g = next_g;
        Part<R, V, NV> res = next_h, d = next_d;
        loaded();
        f2 sq = f2_both(0.0f), ip = f2_both(0.0f);
        // the sum again as the forward pass has it, twice: it is not kept
        auto sum_of = [&](const f2 (&sc)[V / 2], int j, int k) {
            return a.scale != nullptr ? f2_fma(sc[k], x.pair(j, k), res.pair(j, k)) : f2_add(x.pair(j, k), res.pair(j, k));
        };
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            f2 wv[V / 2], sc[V / 2];
            w.load(wv, j);
            if (a.scale != nullptr) scale.load(sc, j);
#pragma unroll
            for (int k = 0; k < V / 2; ++k) {
                const f2 h = sum_of(sc, j, k);
                sq = f2_fma(h, h, sq);
                ip = f2_fma(f2_mul(g.pair(j, k), wv[k]), h, ip);
            }
        }
        float sum[2] = {f2_sum(sq), f2_sum(ip)};
        sum_group<CTA>(sum, a.tg);
        const float rs = rstd_of(sum[0], a);
        const f2 r = f2_both(rs), back = f2_both(-rs * rs * sum[1] / (float)a.width);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            f2 wv[V / 2], sc[V / 2];
            w.load(wv, j);
            if (a.scale != nullptr) scale.load(sc, j);
#pragma unroll
            for (int k = 0; k < V / 2; ++k) {
                const f2 h = sum_of(sc, j, k), gv = g.pair(j, k);
                const f2 dh = f2_fma(r, f2_fma(gv, wv[k], f2_mul(h, back)), d.pair(j, k));
                dw.v[j][k] = f2_fma(gv, f2_mul(h, r), dw.v[j][k]);
                if (a.scale != nullptr) {
                    ds.v[j][k] = f2_fma(dh, x.pair(j, k), ds.v[j][k]);
                    x.set(j, k, f2_mul(sc[k], dh));
                } else {
                    x.set(j, k, dh);
                }
                d.set(j, k, dh);
            }
        }
        if (on) {
            x.store(a.dx, row * a.dx_stride + s.col0, s.lane, a.tg, a.width);
            d.store(a.dresidual, row * a.dresidual_stride + s.col0, s.lane, a.tg, a.width);
        }
    });
    dw.put(a, s, 0, dynamic);
    if (a.scale != nullptr) ds.put(a, s, 1, dynamic);
}

// Weight gradients over the CTAs: eight columns a CTA (a sector of a row of parts),
// 128 threads to a column.  1216 parts of 1024 columns 5.2 us
// (32 columns a CTA, 32 threads each: 8.4).
constexpr int kJoinThreads = 1024, kJoinCols = 8, kSlices = kJoinThreads / kJoinCols;
struct NormJoin {
    const float* parts;
    int n_parts, channels;
    float* out[2];
};
__global__ void __launch_bounds__(kJoinThreads) norm_join_kernel(const __grid_constant__ NormJoin a) {
    __shared__ float red[kJoinThreads / 32][kJoinCols + 1];
    pdl_wait();
    float* out = a.out[blockIdx.y];
    if (out == nullptr) return;
    const int c0 = blockIdx.x * kJoinCols, col = threadIdx.x % kJoinCols, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float* p = a.parts + (int64_t)blockIdx.y * a.n_parts * a.channels + c0 + col;      // channels are eights
    float v = 0.0f;
#pragma unroll 8
    for (int j = threadIdx.x / kJoinCols; j < a.n_parts; j += kSlices) v += p[(int64_t)j * a.channels];
#pragma unroll
    for (int o = kJoinCols; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane < kJoinCols) red[warp][lane] = v;
    __syncthreads();
    if (warp >= kJoinCols) return;
    v = red[lane][warp];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) out[c0 + warp] = v;
}

// fn<.., NV, CTA> for a cut: a CTA's threads have `cta` vectors each, a lane one,
// two, four or eight, up to `most`.
#define OFRL_NORM_PICK(c, cta_nv, most, fn, ...)                                                                   \
    ((c).cta       ? fn<__VA_ARGS__, cta_nv, true>                                                                 \
     : (c).nv == 1 ? fn<__VA_ARGS__, 1, false>                                                                     \
     : (c).nv == 2 ? fn<__VA_ARGS__, 2, false>                                                                     \
     : (c).nv == 4 ? fn<__VA_ARGS__, most < 4 ? most : 4, false>                                                   \
                   : fn<__VA_ARGS__, most, false>)

using NormKernel = void (*)(NormArgs);

// CTAs over rows: what the GPU holds at once, no more than there is work.
int rows_grid(int64_t rows, const NormCut& c, int groups, int num_sms, int per_sm, bool backward) {
    int64_t all = (rows + c.groups_at_once - 1) / c.groups_at_once;
    // a CTA's parts of the weights' gradients cost as much as a row or two
    if (backward && all > num_sms) all = all / 4 > num_sms ? all / 4 : num_sms;
    int64_t most = ((int64_t)num_sms * per_sm + groups - 1) / groups;
    if (most > kMaxParts) most = kMaxParts;
    return (int)(all < 1 ? 1 : all < most ? all : most);
}

NormKernel forward_kernel(const ofrl_norm_shape& s, const NormCut& c, bool gated) {
    const bool f = s.dtype == OFRL_DTYPE_F32, rf = s.residual_dtype == OFRL_DTYPE_F32;
    if (gated)
        return f ? OFRL_NORM_PICK(c, 4, 8, gated_norm_kernel, float) : OFRL_NORM_PICK(c, 2, 4, gated_norm_kernel, __nv_bfloat16);
    if (f) return OFRL_NORM_PICK(c, 4, 8, residual_norm_kernel, float, float);
    return rf ? OFRL_NORM_PICK(c, 2, 4, residual_norm_kernel, __nv_bfloat16, float)
              : OFRL_NORM_PICK(c, 2, 4, residual_norm_kernel, __nv_bfloat16, __nv_bfloat16);
}
NormKernel backward_kernel(const ofrl_norm_shape& s, const NormCut& c, bool gated) {
    const bool f = s.dtype == OFRL_DTYPE_F32, rf = s.residual_dtype == OFRL_DTYPE_F32;
    if (gated)
        return f ? OFRL_NORM_PICK(c, 4, 4, gated_norm_grad_kernel, float)
                 : OFRL_NORM_PICK(c, 2, 2, gated_norm_grad_kernel, __nv_bfloat16);
    if (f) return OFRL_NORM_PICK(c, 4, 4, residual_norm_grad_kernel, float, float);
    return rf ? OFRL_NORM_PICK(c, 2, 2, residual_norm_grad_kernel, __nv_bfloat16, float)
              : OFRL_NORM_PICK(c, 2, 2, residual_norm_grad_kernel, __nv_bfloat16, __nv_bfloat16);
}

NormCut cut_of(const ofrl_norm_shape& s, bool backward) {
    return norm_cut(s.channels / s.groups, (int)dtype_size(s.dtype), backward);
}
// Shared memory of a launch: weights and scales, later (gradients) a row a seat.
int shared_of(const ofrl_norm_shape& s, const NormCut& c) {
    const int row = weight_floats(c.tg, c.nv, 16 / (int)dtype_size(s.dtype));
    return 4 * row * (c.groups_at_once > 2 ? c.groups_at_once : 2);
}

cudaError_t launch_rows(const ofrl_norm_shape& s, bool gated, bool backward, const NormArgs& a, const NormCut& c, int grid,
                        cudaStream_t st) {
    NormKernel k = backward ? backward_kernel(s, c, gated) : forward_kernel(s, c, gated);
    return launch_pdl(k, dim3((unsigned)grid, (unsigned)s.groups), dim3(c.threads), (size_t)shared_of(s, c), st, a);
}

ofrl_status check_shape(const ofrl_norm_shape* s) {
    if (s == nullptr || s->channels < 1 || s->groups < 1 || s->channels % s->groups != 0 || !dtype_ok(s->dtype) ||
        (s->residual_dtype != OFRL_DTYPE_F32 && s->residual_dtype != s->dtype))
        return OFRL_EINVAL;
    const int width = s->channels / s->groups;
    if (s->channels > 65536 || width % 8 != 0 || width > 8192) return OFRL_EUNSUPPORTED;
    return OFRL_OK;
}

bool size_ok(int64_t rows, float eps) { return rows >= 0 && rows <= INT32_MAX && eps > 0.0f && eps < INFINITY; }
bool weights_ok(const float* weight, const float* scale) {
    return weight != nullptr && aligned_to(weight, 16) && aligned_to(scale, 16);
}

ofrl_status check_gated(const ofrl_norm* ctx, const ofrl_gated_rows* in) {
    const ofrl_status s = check_device(ctx);
    if (s != OFRL_OK) return s;
    if (in == nullptr || !size_ok(in->rows, in->eps) || !weights_ok(in->weight, nullptr) ||
        (in->gate_first != 0 && in->gate_first != 1))
        return OFRL_EINVAL;
    const int64_t d = ctx->shape.channels, e = dtype_size(ctx->shape.dtype);
    if (in->rows > 0 && (!rows_ok(in->x, in->x_stride, d, e) || !rows_ok(in->z, in->z_stride, d, e))) return OFRL_EINVAL;
    return OFRL_OK;
}
ofrl_status check_residual(const ofrl_norm* ctx, const ofrl_residual_rows* in) {
    const ofrl_status s = check_device(ctx);
    if (s != OFRL_OK) return s;
    if (in == nullptr || !size_ok(in->rows, in->eps) || !weights_ok(in->weight, in->scale)) return OFRL_EINVAL;
    const int64_t d = ctx->shape.channels, e = dtype_size(ctx->shape.dtype), re = dtype_size(ctx->shape.residual_dtype);
    if (in->rows > 0 && (!rows_ok(in->x, in->x_stride, d, e) || !rows_ok(in->residual, in->residual_stride, d, re)))
        return OFRL_EINVAL;
    return OFRL_OK;
}

NormArgs base_args(const ofrl_norm* ctx) {
    NormArgs a;
    std::memset(&a, 0, sizeof(a));
    a.channels = ctx->shape.channels;
    a.width = ctx->shape.channels / ctx->shape.groups;
    a.parts = ctx->parts;
    return a;
}
NormArgs args_of(const ofrl_norm* ctx, const ofrl_gated_rows* in) {
    NormArgs a = base_args(ctx);
    a.x = in->x;
    a.z = in->z;
    a.weight = in->weight;
    a.x_stride = in->x_stride;
    a.z_stride = in->z_stride;
    a.rows = in->rows;
    a.eps = in->eps;
    a.gate_first = in->gate_first;
    return a;
}
NormArgs args_of(const ofrl_norm* ctx, const ofrl_residual_rows* in) {
    NormArgs a = base_args(ctx);
    a.x = in->x;
    a.residual = in->residual;
    a.scale = in->scale;
    a.weight = in->weight;
    a.x_stride = in->x_stride;
    a.residual_stride = in->residual_stride;
    a.rows = in->rows;
    a.eps = in->eps;
    return a;
}

// How a call is cut, and its CTAs over rows.
struct NormPlan {
    NormCut cut;
    int grid;
};
NormPlan plan_of(const ofrl_norm* ctx, int64_t rows, bool gated, bool backward) {
    NormPlan p;
    p.cut = cut_of(ctx->shape, backward);
    p.grid = rows_grid(rows, p.cut, ctx->shape.groups, ctx->num_sms, ctx->per_sm[gated][backward], backward);
    return p;
}

ofrl_status run_forward(const ofrl_norm* ctx, NormArgs& a, bool gated, cudaStream_t st) {
    if (a.rows == 0) return OFRL_OK;
    const NormPlan p = plan_of(ctx, a.rows, gated, false);
    a.tg = p.cut.tg;
    return cuda_status(launch_rows(ctx->shape, gated, false, a, p.cut, p.grid, st));
}
ofrl_status run_backward(const ofrl_norm* ctx, NormArgs& a, bool gated, float* dweight, float* dscale, cudaStream_t st) {
    const NormPlan p = plan_of(ctx, a.rows, gated, true);
    a.tg = p.cut.tg;
    cudaError_t e = launch_rows(ctx->shape, gated, true, a, p.cut, p.grid, st);
    if (e == cudaSuccess) {
        NormJoin j;
        j.parts = a.parts;
        j.n_parts = p.grid;
        j.channels = a.channels;
        j.out[0] = dweight;
        j.out[1] = dscale;
        e = launch_pdl(norm_join_kernel, dim3((unsigned)(a.channels / kJoinCols), dscale != nullptr ? 2u : 1u),
                       dim3(kJoinThreads), 0, st, j);
    }
    return cuda_status(e);
}

// The workspace: parts of as many CTAs as any backward call has.
int64_t norm_bytes(const ofrl_norm_shape& s, int num_sms, const int (&per_sm)[2][2], bool backward) {
    if (!backward) return 256;
    const int most = per_sm[0][1] > per_sm[1][1] ? per_sm[0][1] : per_sm[1][1];
    return 256 + 2 * (int64_t)rows_grid(INT32_MAX, cut_of(s, true), s.groups, num_sms, most, true) * s.channels * 4;
}
// CTAs of each kernel that an SM holds; opts the kernels into their shared memory.
cudaError_t find_per_sm(const ofrl_norm_shape& s, int (&per_sm)[2][2]) {
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < 4; ++i) {
        const bool gated = i & 1, back = i & 2;
        const NormCut c = cut_of(s, back);
        NormKernel k = back ? backward_kernel(s, c, gated) : forward_kernel(s, c, gated);
        int& n = per_sm[gated][back];
        if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared);
        if (e == cudaSuccess) e = set_max_shared_carveout(k);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k, c.threads, (size_t)shared_of(s, c));
        if (n < 1) n = 1;
    }
    return e;
}

}  // namespace
}  // namespace ofrl

using namespace ofrl;

extern "C" {

int64_t ofrl_norm_workspace_bytes(const ofrl_norm_shape* shape, int32_t backward) {
    if (check_shape(shape) != OFRL_OK || (backward != 0 && backward != 1)) return -1;
    int device = 0, per_sm[2][2] = {};
    int sms = current_sms(&device);
    if (sms == 0 || find_per_sm(*shape, per_sm) != cudaSuccess) {      // no GPU to be asked: one SM, one CTA
        cudaGetLastError();
        sms = 1;
        for (int i = 0; i < 4; ++i) per_sm[i & 1][i >> 1] = 1;
    }
    return norm_bytes(*shape, sms, per_sm, backward != 0);
}

ofrl_status ofrl_norm_create(const ofrl_norm_shape* shape, int32_t backward, ofrl_norm** out) {
    if (out == nullptr) return OFRL_EINVAL;
    *out = nullptr;
    const ofrl_status s = check_shape(shape);
    if (s != OFRL_OK) return s;
    if (backward != 0 && backward != 1) return OFRL_EINVAL;
    ofrl_norm* ctx = new (std::nothrow) ofrl_norm;
    if (ctx == nullptr) return OFRL_ECUDA;
    std::memset(ctx, 0, sizeof(*ctx));
    ctx->num_sms = current_sms(&ctx->device);
    ctx->shape = *shape;
    ctx->backward = backward;
    if (ctx->num_sms == 0 || find_per_sm(*shape, ctx->per_sm) != cudaSuccess) {
        cudaGetLastError();
        delete ctx;
        return OFRL_ECUDA;
    }
    ctx->bytes = norm_bytes(*shape, ctx->num_sms, ctx->per_sm, backward != 0);
    if (take_memory(&ctx->base, ctx->bytes) != cudaSuccess) {
        delete ctx;
        return OFRL_ECUDA;
    }
    ctx->parts = reinterpret_cast<float*>(static_cast<char*>(ctx->base) + 256);
    *out = ctx;
    return OFRL_OK;
}

ofrl_status ofrl_norm_destroy(ofrl_norm* ctx) { return release_memory(ctx); }

ofrl_status ofrl_gated_norm(ofrl_norm* ctx, const ofrl_gated_rows* in, void* out, int64_t out_stride, void* stream) {
    const ofrl_status s = check_gated(ctx, in);
    if (s != OFRL_OK) return s;
    if (in->rows > 0 && !rows_ok(out, out_stride, ctx->shape.channels, dtype_size(ctx->shape.dtype))) return OFRL_EINVAL;
    NormArgs a = args_of(ctx, in);
    a.out = out;
    a.out_stride = out_stride;
    return run_forward(ctx, a, true, static_cast<cudaStream_t>(stream));
}

ofrl_status ofrl_gated_norm_backward(ofrl_norm* ctx, const ofrl_gated_rows* in, const void* dout, int64_t dout_stride,
                                     void* dx, int64_t dx_stride, void* dz, int64_t dz_stride, float* dweight,
                                     void* stream) {
    const ofrl_status s = check_gated(ctx, in);
    if (s != OFRL_OK) return s;
    if (!ctx->backward || dweight == nullptr || !aligned_to(dweight, 4)) return OFRL_EINVAL;
    const int64_t d = ctx->shape.channels, e = dtype_size(ctx->shape.dtype);
    if (in->rows > 0 &&
        (!rows_ok(dout, dout_stride, d, e) || !rows_ok(dx, dx_stride, d, e) || !rows_ok(dz, dz_stride, d, e)))
        return OFRL_EINVAL;
    NormArgs a = args_of(ctx, in);
    a.dout = dout;
    a.dout_stride = dout_stride;
    a.dx = dx;
    a.dx_stride = dx_stride;
    a.dz = dz;
    a.dz_stride = dz_stride;
    return run_backward(ctx, a, true, dweight, nullptr, static_cast<cudaStream_t>(stream));
}

ofrl_status ofrl_residual_norm(ofrl_norm* ctx, const ofrl_residual_rows* in, void* residual_out,
                               int64_t residual_out_stride, void* out, int64_t out_stride, void* stream) {
    const ofrl_status s = check_residual(ctx, in);
    if (s != OFRL_OK) return s;
    const int64_t d = ctx->shape.channels;
    if (in->rows > 0 && (!rows_ok(out, out_stride, d, dtype_size(ctx->shape.dtype)) ||
                         !rows_ok(residual_out, residual_out_stride, d, dtype_size(ctx->shape.residual_dtype))))
        return OFRL_EINVAL;
    NormArgs a = args_of(ctx, in);
    a.residual_out = residual_out;
    a.residual_out_stride = residual_out_stride;
    a.out = out;
    a.out_stride = out_stride;
    return run_forward(ctx, a, false, static_cast<cudaStream_t>(stream));
}

ofrl_status ofrl_residual_norm_backward(ofrl_norm* ctx, const ofrl_residual_rows* in, const void* dout,
                                        int64_t dout_stride, const void* d_residual_out, int64_t d_residual_out_stride,
                                        void* dx, int64_t dx_stride, void* dresidual, int64_t dresidual_stride,
                                        float* dweight, float* dscale, void* stream) {
    const ofrl_status s = check_residual(ctx, in);
    if (s != OFRL_OK) return s;
    if (!ctx->backward || dweight == nullptr || !aligned_to(dweight, 4) || !aligned_to(dscale, 4) ||
        (dscale == nullptr) != (in->scale == nullptr))
        return OFRL_EINVAL;
    const int64_t d = ctx->shape.channels, e = dtype_size(ctx->shape.dtype), re = dtype_size(ctx->shape.residual_dtype);
    if (in->rows > 0 && (!rows_ok(dout, dout_stride, d, e) || !rows_ok(dx, dx_stride, d, e) ||
                         !rows_ok(dresidual, dresidual_stride, d, re) ||
                         (d_residual_out != nullptr && !rows_ok(d_residual_out, d_residual_out_stride, d, re))))
        return OFRL_EINVAL;
    NormArgs a = args_of(ctx, in);
    a.dout = dout;
    a.dout_stride = dout_stride;
    a.dres = d_residual_out;
    a.dres_stride = d_residual_out_stride;
    a.dx = dx;
    a.dx_stride = dx_stride;
    a.dresidual = dresidual;
    a.dresidual_stride = dresidual_stride;
    return run_backward(ctx, a, false, dweight, dscale, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
