// Norms around a block: the gated norm after its memory and the norm of the
// residual stream before the next block; forward and gradients.
//
// With s = 1 / rms(u) over a group of W channels, e = dout (times the gate where
// it comes after the norm) and c = sum(e w u) / W:
//   out = w u s          du = s (e w - u s^2 c)          dw = sum over rows of e u s
// u is x, x silu(z), or h = residual + scale x.  Both sums of a row (u^2 and
// e w u) come from one read of it, which stays in registers until its outputs
// are written, so each tensor moves once.  Bound by HBM.
//
// A group of channels has up to 32 lanes of a warp, or a whole CTA.  Threads keep their columns over the rows they take, so
// a weight's gradient is a register until the end; then it is added over the
// CTA, and by a second launch over the CTAs, in a fixed order.

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

// What a launch's threads are to its rows.  A thread has eight elements of a row,
// so that these, the next row's and a weight's gradient stay in registers; rows
// of more than 4096 channels have sixteen, and no row ahead.
struct NormCut {
    bool cta;
    int threads, tg, nv, groups_at_once;
};
NormCut norm_cut(int width, int elem) {
    const int vecs = width * elem / 16, usual = elem == 2 ? 1 : 2;
    NormCut c;
    c.cta = vecs > 32 * usual;
    c.tg = c.cta ? 64 : 1;
    while (c.cta ? c.tg < 512 && c.tg * usual < vecs : c.tg < 32 && c.tg < vecs) c.tg *= 2;
    c.threads = c.cta ? c.tg : kWarpThreads;
    const int nv = (vecs + c.tg - 1) / c.tg;
    c.nv = nv <= 1 ? 1 : nv <= 2 ? 2 : 4;
    c.groups_at_once = c.threads / c.tg;
    return c;
}

// Sums of a and b over the group's threads, to all of them.
template <bool CTA>
__device__ __forceinline__ void sum_group(float& a, float& b, int tg) {
    if constexpr (!CTA) {
        for (int o = tg >> 1; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
    } else {
        __shared__ float2 p[16];
        a = warp_sum(a);
        b = warp_sum(b);
        __syncthreads();          // the row before has read its sums
        if ((threadIdx.x & 31) == 0) p[threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        a = b = 0.0f;
        for (int i = 0; i < tg / 32; ++i) {
            a += p[i].x;
            b += p[i].y;
        }
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

// Rows go by with the next one's loads in flight where AHEAD: fetch(row, on)
// loads, body(row, on) starts with a copy of what was loaded and then calls the
// function it is given.
template <bool AHEAD, bool CTA, typename Fetch, typename Body>
__device__ __forceinline__ void for_rows(const NormArgs& a, const Seat<CTA>& s, const Fetch& fetch, const Body& body) {
    const int64_t step = (int64_t)gridDim.x * s.at_once;
    int64_t row0 = (int64_t)blockIdx.x * s.at_once;
    if (AHEAD) fetch(row0 + s.seat, row0 + s.seat < a.rows);
    for (; row0 < a.rows; row0 += step) {
        const int64_t row = row0 + s.seat, after = row + step;
        if (!AHEAD) fetch(row, row < a.rows);
        body(row, row < a.rows, [&]() {
            if (AHEAD) fetch(after, after < a.rows);
        });
    }
}
template <typename T, int NV>
constexpr bool kRowAhead = NV * kVec<T> <= 8;

template <typename T, int NV, bool CTA>
__global__ void __launch_bounds__(CTA ? 512 : kWarpThreads) gated_norm_kernel(const __grid_constant__ NormArgs a) {
    constexpr int V = kVec<T>;
    pdl_wait();
    pdl_trigger();
    const Seat<CTA> s(a);
    Part<float, V, NV> w;
    w.load(a.weight, s.col0, s.lane, a.tg, a.width, true);
    Part<T, V, NV> next_x, next_z;
    auto fetch = [&](int64_t row, bool on) {
        next_x.load(a.x, row * a.x_stride + s.col0, s.lane, a.tg, a.width, on);
        next_z.load(a.z, row * a.z_stride + s.col0, s.lane, a.tg, a.width, on);
    };
    for_rows<kRowAhead<T, NV>>(a, s, fetch, [&](int64_t row, bool on, auto loaded) {
        Part<T, V, NV> x = next_x, z = next_z;
        loaded();
        f2 u[NV][V / 2], g[NV][V / 2], sq = f2_both(0.0f);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < V / 2; ++k) {
                u[j][k] = x.pair(j, k);
                g[j][k] = silu(z.pair(j, k));
                if (a.gate_first) {
                    u[j][k] = f2_mul(u[j][k], g[j][k]);
                    g[j][k] = w.pair(j, k);
                } else {
                    g[j][k] = f2_mul(g[j][k], w.pair(j, k));
                }
                sq = f2_fma(u[j][k], u[j][k], sq);
            }
        float sum = f2_sum(sq), none = 0.0f;
        sum_group<CTA>(sum, none, a.tg);
        const f2 r = f2_both(rstd_of(sum, a));
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < V / 2; ++k) x.set(j, k, f2_mul(f2_mul(u[j][k], r), g[j][k]));
        if (on) x.store(a.out, row * a.out_stride + s.col0, s.lane, a.tg, a.width);
    });
}

// T: x and out, R: the residual.
template <typename T, typename R, int NV, bool CTA>
__global__ void __launch_bounds__(CTA ? 512 : kWarpThreads) residual_norm_kernel(const __grid_constant__ NormArgs a) {
    constexpr int V = kVec<T>;
    pdl_wait();
    pdl_trigger();
    const Seat<CTA> s(a);
    Part<float, V, NV> w, scale;
    w.load(a.weight, s.col0, s.lane, a.tg, a.width, true);
    if (a.scale != nullptr) scale.load(a.scale, s.col0, s.lane, a.tg, a.width, true);
    Part<T, V, NV> next_x;
    Part<R, V, NV> next_h;
    auto fetch = [&](int64_t row, bool on) {
        next_x.load(a.x, row * a.x_stride + s.col0, s.lane, a.tg, a.width, on);
        next_h.load(a.residual, row * a.residual_stride + s.col0, s.lane, a.tg, a.width, on);
    };
    for_rows<kRowAhead<T, NV>>(a, s, fetch, [&](int64_t row, bool on, auto loaded) {
        Part<T, V, NV> x = next_x;
        Part<R, V, NV> res = next_h;
        loaded();
        f2 h[NV][V / 2], sq = f2_both(0.0f);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < V / 2; ++k) {
                h[j][k] = a.scale != nullptr ? f2_fma(scale.pair(j, k), x.pair(j, k), res.pair(j, k))
                                             : f2_add(x.pair(j, k), res.pair(j, k));
                sq = f2_fma(h[j][k], h[j][k], sq);
                res.set(j, k, h[j][k]);
            }
        if (on) res.store(a.residual_out, row * a.residual_out_stride + s.col0, s.lane, a.tg, a.width);
        float sum = f2_sum(sq), none = 0.0f;
        sum_group<CTA>(sum, none, a.tg);
        const f2 r = f2_both(rstd_of(sum, a));
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < V / 2; ++k) x.set(j, k, f2_mul(f2_mul(h[j][k], r), w.pair(j, k)));
        if (on) x.store(a.out, row * a.out_stride + s.col0, s.lane, a.tg, a.width);
    });
}

// A column's gradient over the CTA's seats, to the CTA's place in parts.
template <int V, int NV, bool CTA>
__device__ __forceinline__ void put_parts(const NormArgs& a, const Seat<CTA>& s, const Part<float, V, NV>& g, int which,
                                          float* red) {
    float* out = a.parts + ((int64_t)which * gridDim.x + blockIdx.x) * a.channels + s.col0;
    if constexpr (CTA) {
        g.store(out, 0, s.lane, a.tg, a.width);
    } else {
        __syncthreads();
        const int row = a.tg * NV * V;
        g.store(red, s.seat * row, s.lane, a.tg, row);
        __syncthreads();
        for (int c = threadIdx.x; c < a.width; c += blockDim.x) {
            float v = 0.0f;
            for (int i = 0; i < s.at_once; ++i) v += red[i * row + c];
            out[c] = v;
        }
    }
}

template <typename T, int NV, bool CTA>
__global__ void __launch_bounds__(CTA ? 512 : kWarpThreads) gated_norm_grad_kernel(const __grid_constant__ NormArgs a) {
    constexpr int V = kVec<T>;
    __shared__ __align__(16) float red[CTA ? 4 : kWarpThreads * NV * V];
    pdl_wait();
    pdl_trigger();
    const Seat<CTA> s(a);
    Part<float, V, NV> w, dw;
    w.load(a.weight, s.col0, s.lane, a.tg, a.width, true);
    dw.load(a.weight, 0, s.lane, a.tg, a.width, false);      // zero
    Part<T, V, NV> next_x, next_z, next_g;
    auto fetch = [&](int64_t row, bool on) {
        next_x.load(a.x, row * a.x_stride + s.col0, s.lane, a.tg, a.width, on);
        next_z.load(a.z, row * a.z_stride + s.col0, s.lane, a.tg, a.width, on);
        next_g.load(a.dout, row * a.dout_stride + s.col0, s.lane, a.tg, a.width, on);
    };
    for_rows<kRowAhead<T, NV>>(a, s, fetch, [&](int64_t row, bool on, auto loaded) {
        Part<T, V, NV> x = next_x, z = next_z, g = next_g;
        loaded();
        f2 sq = f2_both(0.0f), ip = f2_both(0.0f);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < V / 2; ++k) {
                const f2 gate = silu(z.pair(j, k));
                f2 u = x.pair(j, k), e = g.pair(j, k);
                if (a.gate_first)
                    u = f2_mul(u, gate);
                else
                    e = f2_mul(e, gate);
                sq = f2_fma(u, u, sq);
                ip = f2_fma(f2_mul(e, w.pair(j, k)), u, ip);
            }
        float sum = f2_sum(sq), dot = f2_sum(ip);
        sum_group<CTA>(sum, dot, a.tg);
        const float rs = rstd_of(sum, a);
        const f2 r = f2_both(rs), back = f2_both(-rs * rs * dot / (float)a.width);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < V / 2; ++k) {
                const f2 zv = z.pair(j, k), sg = sigmoid(zv), gate = f2_mul(zv, sg), wv = w.pair(j, k), xv = x.pair(j, k);
                f2 u = xv, e = g.pair(j, k), dgate;
                if (a.gate_first)
                    u = f2_mul(u, gate);
                else
                    e = f2_mul(e, gate);
                const f2 unit = f2_mul(u, r), du = f2_mul(r, f2_fma(e, wv, f2_mul(u, back)));
                dw.set(j, k, f2_fma(e, unit, dw.pair(j, k)));
                dgate = a.gate_first ? f2_mul(du, xv) : f2_mul(f2_mul(g.pair(j, k), unit), wv);
                x.set(j, k, a.gate_first ? f2_mul(du, gate) : du);
                z.set(j, k, f2_mul(dgate, silu_slope(zv, sg)));
            }
        if (on) {
            x.store(a.dx, row * a.dx_stride + s.col0, s.lane, a.tg, a.width);
            z.store(a.dz, row * a.dz_stride + s.col0, s.lane, a.tg, a.width);
        }
    });
    put_parts<V, NV, CTA>(a, s, dw, 0, red);
}

template <typename T, typename R, int NV, bool CTA>
__global__ void __launch_bounds__(CTA ? 512 : kWarpThreads) residual_norm_grad_kernel(const __grid_constant__ NormArgs a) {
    constexpr int V = kVec<T>;
    __shared__ __align__(16) float red[CTA ? 4 : kWarpThreads * NV * V];
    pdl_wait();
    pdl_trigger();
    const Seat<CTA> s(a);
    Part<float, V, NV> w, scale, dw, ds;
    w.load(a.weight, s.col0, s.lane, a.tg, a.width, true);
    if (a.scale != nullptr) scale.load(a.scale, s.col0, s.lane, a.tg, a.width, true);
    dw.load(a.weight, 0, s.lane, a.tg, a.width, false);      // zero
    ds.load(a.weight, 0, s.lane, a.tg, a.width, false);
    Part<T, V, NV> next_x, next_g;
    Part<R, V, NV> next_h, next_d;
    auto fetch = [&](int64_t row, bool on) {
        next_x.load(a.x, row * a.x_stride + s.col0, s.lane, a.tg, a.width, on);
        next_h.load(a.residual, row * a.residual_stride + s.col0, s.lane, a.tg, a.width, on);
        next_g.load(a.dout, row * a.dout_stride + s.col0, s.lane, a.tg, a.width, on);
        next_d.load(a.dres, row * a.dres_stride + s.col0, s.lane, a.tg, a.width, on && a.dres != nullptr);
    };
    for_rows<kRowAhead<T, NV>>(a, s, fetch, [&](int64_t row, bool on, auto loaded) {
        Part<T, V, NV> x = next_x, g = next_g;
        Part<R, V, NV> res = next_h, d = next_d;
        loaded();
        f2 h[NV][V / 2], sq = f2_both(0.0f), ip = f2_both(0.0f);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < V / 2; ++k) {
                h[j][k] = a.scale != nullptr ? f2_fma(scale.pair(j, k), x.pair(j, k), res.pair(j, k))
                                             : f2_add(x.pair(j, k), res.pair(j, k));
                sq = f2_fma(h[j][k], h[j][k], sq);
                ip = f2_fma(f2_mul(g.pair(j, k), w.pair(j, k)), h[j][k], ip);
            }
        float sum = f2_sum(sq), dot = f2_sum(ip);
        sum_group<CTA>(sum, dot, a.tg);
        const float rs = rstd_of(sum, a);
        const f2 r = f2_both(rs), back = f2_both(-rs * rs * dot / (float)a.width);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < V / 2; ++k) {
                const f2 gv = g.pair(j, k), dh = f2_fma(r, f2_fma(gv, w.pair(j, k), f2_mul(h[j][k], back)), d.pair(j, k));
                dw.set(j, k, f2_fma(gv, f2_mul(h[j][k], r), dw.pair(j, k)));
                if (a.scale != nullptr) {
                    ds.set(j, k, f2_fma(dh, x.pair(j, k), ds.pair(j, k)));
                    x.set(j, k, f2_mul(scale.pair(j, k), dh));
                } else {
                    x.set(j, k, dh);
                }
                d.set(j, k, dh);
            }
        if (on) {
            x.store(a.dx, row * a.dx_stride + s.col0, s.lane, a.tg, a.width);
            d.store(a.dresidual, row * a.dresidual_stride + s.col0, s.lane, a.tg, a.width);
        }
    });
    put_parts<V, NV, CTA>(a, s, dw, 0, red);
    if (a.scale != nullptr) put_parts<V, NV, CTA>(a, s, ds, 1, red);
}

// Weight gradients over the CTAs: 32 columns a CTA, 32 threads to a column.
constexpr int kJoinThreads = 1024, kSlices = kJoinThreads / 32;
struct NormJoin {
    const float* parts;
    int n_parts, channels;
    float* out[2];
};
__global__ void __launch_bounds__(kJoinThreads) norm_join_kernel(const __grid_constant__ NormJoin a) {
    __shared__ float red[kSlices][33];
    pdl_wait();
    pdl_trigger();
    const int c = blockIdx.x * 32 + threadIdx.x % 32, slice = threadIdx.x / 32;
    float* out = a.out[blockIdx.y];
    if (out == nullptr) return;
    const float* p = a.parts + (int64_t)blockIdx.y * a.n_parts * a.channels;
    float v = 0.0f;
    if (c < a.channels) {
#pragma unroll 8
        for (int j = slice; j < a.n_parts; j += kSlices) v += p[(int64_t)j * a.channels + c];
    }
    red[slice][threadIdx.x % 32] = v;
    __syncthreads();
    if (slice > 0 || c >= a.channels) return;
    v = 0.0f;
    for (int k = 0; k < kSlices; ++k) v += red[k][threadIdx.x];
    out[c] = v;
}

// fn<.., NV, CTA> for a cut (bf16 rows never have four vectors a thread).
#define OFRL_NORM_PICK(c, fn, ...)                                                                                 \
    ((c).cta ? ((c).nv == 1 ? fn<__VA_ARGS__, 1, true> : fn<__VA_ARGS__, 2, true>)                                 \
             : ((c).nv == 1 ? fn<__VA_ARGS__, 1, false> : fn<__VA_ARGS__, 2, false>))
#define OFRL_NORM_PICK4(c, fn, ...)                                                                                \
    ((c).nv < 4 ? OFRL_NORM_PICK(c, fn, __VA_ARGS__) : (c).cta ? fn<__VA_ARGS__, 4, true> : fn<__VA_ARGS__, 4, false>)

using NormKernel = void (*)(NormArgs);

// CTAs over rows: what the GPU holds at once, no more than there is work.
int rows_grid(int64_t rows, const NormCut& c, int groups, int num_sms, int per_sm) {
    const int64_t all = (rows + c.groups_at_once - 1) / c.groups_at_once;
    int64_t most = ((int64_t)num_sms * per_sm + groups - 1) / groups;
    if (most > kMaxParts) most = kMaxParts;
    return (int)(all < 1 ? 1 : all < most ? all : most);
}

cudaError_t launch_rows(NormKernel kernel, const NormArgs& a, const NormCut& c, int groups, int grid, cudaStream_t st) {
    return launch_pdl(kernel, dim3((unsigned)grid, (unsigned)groups), dim3(c.threads), 0, st, a);
}

NormKernel forward_kernel(const ofrl_norm_shape& s, const NormCut& c, bool gated) {
    const bool f = s.dtype == OFRL_DTYPE_F32, rf = s.residual_dtype == OFRL_DTYPE_F32;
    if (gated) return f ? OFRL_NORM_PICK4(c, gated_norm_kernel, float) : OFRL_NORM_PICK(c, gated_norm_kernel, __nv_bfloat16);
    if (f) return OFRL_NORM_PICK4(c, residual_norm_kernel, float, float);
    return rf ? OFRL_NORM_PICK(c, residual_norm_kernel, __nv_bfloat16, float)
              : OFRL_NORM_PICK(c, residual_norm_kernel, __nv_bfloat16, __nv_bfloat16);
}
NormKernel backward_kernel(const ofrl_norm_shape& s, const NormCut& c, bool gated) {
    const bool f = s.dtype == OFRL_DTYPE_F32, rf = s.residual_dtype == OFRL_DTYPE_F32;
    if (gated)
        return f ? OFRL_NORM_PICK4(c, gated_norm_grad_kernel, float) : OFRL_NORM_PICK(c, gated_norm_grad_kernel, __nv_bfloat16);
    if (f) return OFRL_NORM_PICK4(c, residual_norm_grad_kernel, float, float);
    return rf ? OFRL_NORM_PICK(c, residual_norm_grad_kernel, __nv_bfloat16, float)
              : OFRL_NORM_PICK(c, residual_norm_grad_kernel, __nv_bfloat16, __nv_bfloat16);
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

NormArgs base_args(const ofrl_norm* ctx, const NormCut& c) {
    NormArgs a;
    std::memset(&a, 0, sizeof(a));
    a.channels = ctx->shape.channels;
    a.width = ctx->shape.channels / ctx->shape.groups;
    a.tg = c.tg;
    a.parts = ctx->parts;
    return a;
}
NormCut cut_of(const ofrl_norm* ctx) {
    return norm_cut(ctx->shape.channels / ctx->shape.groups, (int)dtype_size(ctx->shape.dtype));
}
NormArgs args_of(const ofrl_norm* ctx, const NormCut& c, const ofrl_gated_rows* in) {
    NormArgs a = base_args(ctx, c);
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
NormArgs args_of(const ofrl_norm* ctx, const NormCut& c, const ofrl_residual_rows* in) {
    NormArgs a = base_args(ctx, c);
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

ofrl_status run_forward(const ofrl_norm* ctx, const NormCut& c, const NormArgs& a, bool gated, cudaStream_t st) {
    if (a.rows == 0) return OFRL_OK;
    const int groups = ctx->shape.groups;
    return cuda_status(launch_rows(forward_kernel(ctx->shape, c, gated), a, c, groups,
                                   rows_grid(a.rows, c, groups, ctx->num_sms, ctx->per_sm[gated][0]), st));
}
ofrl_status run_backward(const ofrl_norm* ctx, const NormCut& c, const NormArgs& a, bool gated, float* dweight,
                         float* dscale, cudaStream_t st) {
    const int groups = ctx->shape.groups, grid = rows_grid(a.rows, c, groups, ctx->num_sms, ctx->per_sm[gated][1]);
    cudaError_t e = launch_rows(backward_kernel(ctx->shape, c, gated), a, c, groups, grid, st);
    if (e == cudaSuccess) {
        NormJoin j;
        j.parts = a.parts;
        j.n_parts = grid;
        j.channels = a.channels;
        j.out[0] = dweight;
        j.out[1] = dscale;
        e = launch_pdl(norm_join_kernel, dim3((unsigned)((a.channels + 31) / 32), dscale != nullptr ? 2u : 1u),
                       dim3(kJoinThreads), 0, st, j);
    }
    return cuda_status(e);
}

int64_t norm_bytes(const ofrl_norm_shape& s, int num_sms, int per_sm, bool backward) {
    if (!backward) return 256;
    const NormCut c = norm_cut(s.channels / s.groups, (int)dtype_size(s.dtype));
    return 256 + 2 * (int64_t)rows_grid(INT32_MAX, c, s.groups, num_sms, per_sm) * s.channels * 4;
}
// CTAs of each kernel that an SM holds.
cudaError_t find_per_sm(const ofrl_norm_shape& s, int (&per_sm)[2][2]) {
    const NormCut c = norm_cut(s.channels / s.groups, (int)dtype_size(s.dtype));
    cudaError_t e = cudaSuccess;
    for (int gated = 0; gated < 2; ++gated)
        for (int back = 0; back < 2; ++back) {
            NormKernel k = back ? backward_kernel(s, c, gated != 0) : forward_kernel(s, c, gated != 0);
            if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm[gated][back], k, c.threads, 0);
            if (per_sm[gated][back] < 1) per_sm[gated][back] = 1;
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
    const int sms = current_sms(&device);
    if (sms == 0 || find_per_sm(*shape, per_sm) != cudaSuccess) {      // no GPU to be asked
        cudaGetLastError();
        return norm_bytes(*shape, 1, 1, backward != 0);
    }
    return norm_bytes(*shape, sms, per_sm[0][1] > per_sm[1][1] ? per_sm[0][1] : per_sm[1][1], backward != 0);
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
    ctx->bytes = norm_bytes(*shape, ctx->num_sms, ctx->per_sm[0][1] > ctx->per_sm[1][1] ? ctx->per_sm[0][1] : ctx->per_sm[1][1],
                            backward != 0);
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
    const NormCut c = cut_of(ctx);
    NormArgs a = args_of(ctx, c, in);
    a.out = out;
    a.out_stride = out_stride;
    return run_forward(ctx, c, a, true, static_cast<cudaStream_t>(stream));
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
    const NormCut c = cut_of(ctx);
    NormArgs a = args_of(ctx, c, in);
    a.dout = dout;
    a.dout_stride = dout_stride;
    a.dx = dx;
    a.dx_stride = dx_stride;
    a.dz = dz;
    a.dz_stride = dz_stride;
    return run_backward(ctx, c, a, true, dweight, nullptr, static_cast<cudaStream_t>(stream));
}

ofrl_status ofrl_residual_norm(ofrl_norm* ctx, const ofrl_residual_rows* in, void* residual_out,
                               int64_t residual_out_stride, void* out, int64_t out_stride, void* stream) {
    const ofrl_status s = check_residual(ctx, in);
    if (s != OFRL_OK) return s;
    const int64_t d = ctx->shape.channels;
    if (in->rows > 0 && (!rows_ok(out, out_stride, d, dtype_size(ctx->shape.dtype)) ||
                         !rows_ok(residual_out, residual_out_stride, d, dtype_size(ctx->shape.residual_dtype))))
        return OFRL_EINVAL;
    const NormCut c = cut_of(ctx);
    NormArgs a = args_of(ctx, c, in);
    a.residual_out = residual_out;
    a.residual_out_stride = residual_out_stride;
    a.out = out;
    a.out_stride = out_stride;
    return run_forward(ctx, c, a, false, static_cast<cudaStream_t>(stream));
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
    const NormCut c = cut_of(ctx);
    NormArgs a = args_of(ctx, c, in);
    a.dout = dout;
    a.dout_stride = dout_stride;
    a.dres = d_residual_out;
    a.dres_stride = d_residual_out_stride;
    a.dx = dx;
    a.dx_stride = dx_stride;
    a.dresidual = dresidual;
    a.dresidual_stride = dresidual_stride;
    return run_backward(ctx, c, a, false, dweight, dscale, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
