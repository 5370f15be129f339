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
// A group of channels has up to 32 lanes of a warp, or a whole CTA, at most 16
// elements a thread.  Threads keep their columns over the rows they take, so
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
};

namespace ofrl {
namespace {

constexpr int kWarpThreads = 128;        // of a CTA that has a warp or less for a group
constexpr int kMaxParts = 2048;          // CTAs over rows of a backward call, at most

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

// Vectors of a thread, at most: 16 elements, which with their gradients and
// weights stay in registers.
constexpr int most_vecs(int elem) { return elem == 2 ? 2 : 4; }

// What a launch's threads are to its rows.
struct NormCut {
    bool cta;
    int threads, tg, nv, groups_at_once;
};
NormCut norm_cut(int width, int elem) {
    const int vecs = width * elem / 16, most = most_vecs(elem);
    NormCut c;
    c.cta = vecs > 32 * most;
    c.tg = c.cta ? 64 : 1;
    while (c.cta ? c.tg * most < vecs : c.tg < 32 && c.tg < vecs) c.tg *= 2;
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

// NV vectors of V elements a thread, zero past the group's width.
template <typename S, int V, int NV>
__device__ __forceinline__ void load_row(float (&v)[NV][V], const void* base, int64_t at, int lane, int tg, int width,
                                         bool on) {
    const S* p = static_cast<const S*>(base) + at;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (lane + j * tg) * V;
        if (on && c < width) {
            if constexpr (V * sizeof(S) == 32) {
                load_vec<S, 4>(*reinterpret_cast<float(*)[4]>(&v[j][0]), p + c);
                load_vec<S, 4>(*reinterpret_cast<float(*)[4]>(&v[j][4]), p + c + 4);
            } else {
                load_vec<S, V>(v[j], p + c);
            }
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) v[j][k] = 0.0f;
        }
    }
}
template <typename S, int V, int NV>
__device__ __forceinline__ void store_row(void* base, int64_t at, const float (&v)[NV][V], int lane, int tg, int width) {
    S* p = static_cast<S*>(base) + at;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (lane + j * tg) * V;
        if (c >= width) continue;
        if constexpr (V * sizeof(S) == 32) {
            store_vec<S, 4>(p + c, *reinterpret_cast<const float(*)[4]>(&v[j][0]));
            store_vec<S, 4>(p + c + 4, *reinterpret_cast<const float(*)[4]>(&v[j][4]));
        } else {
            store_vec<S, V>(p + c, v[j]);
        }
    }
}

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

template <typename T, int NV, bool CTA>
__global__ void __launch_bounds__(CTA ? 512 : kWarpThreads) gated_norm_kernel(const __grid_constant__ NormArgs a) {
    constexpr int V = kVec<T>;
    pdl_wait();
    pdl_trigger();
    const Seat<CTA> s(a);
    float w[NV][V];
    load_row<float, V, NV>(w, a.weight, s.col0, s.lane, a.tg, a.width, true);
    for (int64_t row0 = (int64_t)blockIdx.x * s.at_once; row0 < a.rows; row0 += (int64_t)gridDim.x * s.at_once) {
        const int64_t row = row0 + s.seat;
        const bool on = row < a.rows;
        float x[NV][V], z[NV][V];
        load_row<T, V, NV>(x, a.x, row * a.x_stride + s.col0, s.lane, a.tg, a.width, on);
        load_row<T, V, NV>(z, a.z, row * a.z_stride + s.col0, s.lane, a.tg, a.width, on);
        float sq = 0.0f, none = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float gate = z[j][k] * sigmoid(z[j][k]);
                if (a.gate_first) x[j][k] *= gate;
                z[j][k] = a.gate_first ? w[j][k] : w[j][k] * gate;
                sq = fmaf(x[j][k], x[j][k], sq);
            }
        sum_group<CTA>(sq, none, a.tg);
        const float r = rstd_of(sq, a);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < V; ++k) x[j][k] = x[j][k] * r * z[j][k];
        if (on) store_row<T, V, NV>(a.out, row * a.out_stride + s.col0, x, s.lane, a.tg, a.width);
    }
}

// T: x and out, R: the residual.
template <typename T, typename R, int NV, bool CTA>
__global__ void __launch_bounds__(CTA ? 512 : kWarpThreads) residual_norm_kernel(const __grid_constant__ NormArgs a) {
    constexpr int V = kVec<T>;
    pdl_wait();
    pdl_trigger();
    const Seat<CTA> s(a);
    float w[NV][V], scale[NV][V];
    load_row<float, V, NV>(w, a.weight, s.col0, s.lane, a.tg, a.width, true);
    if (a.scale != nullptr) load_row<float, V, NV>(scale, a.scale, s.col0, s.lane, a.tg, a.width, true);
    for (int64_t row0 = (int64_t)blockIdx.x * s.at_once; row0 < a.rows; row0 += (int64_t)gridDim.x * s.at_once) {
        const int64_t row = row0 + s.seat;
        const bool on = row < a.rows;
        float x[NV][V], h[NV][V];
        load_row<T, V, NV>(x, a.x, row * a.x_stride + s.col0, s.lane, a.tg, a.width, on);
        load_row<R, V, NV>(h, a.residual, row * a.residual_stride + s.col0, s.lane, a.tg, a.width, on);
        float sq = 0.0f, none = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                h[j][k] = a.scale != nullptr ? fmaf(scale[j][k], x[j][k], h[j][k]) : h[j][k] + x[j][k];
                sq = fmaf(h[j][k], h[j][k], sq);
            }
        if (on) store_row<R, V, NV>(a.residual_out, row * a.residual_out_stride + s.col0, h, s.lane, a.tg, a.width);
        sum_group<CTA>(sq, none, a.tg);
        const float r = rstd_of(sq, a);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < V; ++k) h[j][k] = h[j][k] * r * w[j][k];
        if (on) store_row<T, V, NV>(a.out, row * a.out_stride + s.col0, h, s.lane, a.tg, a.width);
    }
}

// A column's gradient over the CTA's seats, to the CTA's place in parts.
template <int V, int NV, bool CTA>
__device__ __forceinline__ void put_parts(const NormArgs& a, const Seat<CTA>& s, float (&g)[NV][V], int which, float* red) {
    float* out = a.parts + ((int64_t)which * gridDim.x + blockIdx.x) * a.channels + s.col0;
    if constexpr (CTA) {
        store_row<float, V, NV>(out, 0, g, s.lane, a.tg, a.width);
    } else {
        __syncthreads();
        const int row = a.tg * NV * V;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < V; ++k) red[s.seat * row + (s.lane + j * a.tg) * V + k] = g[j][k];
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
    __shared__ float red[CTA ? 1 : kWarpThreads * NV * V];
    pdl_wait();
    pdl_trigger();
    const Seat<CTA> s(a);
    float w[NV][V], dw[NV][V];
    load_row<float, V, NV>(w, a.weight, s.col0, s.lane, a.tg, a.width, true);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < V; ++k) dw[j][k] = 0.0f;
    for (int64_t row0 = (int64_t)blockIdx.x * s.at_once; row0 < a.rows; row0 += (int64_t)gridDim.x * s.at_once) {
        const int64_t row = row0 + s.seat;
        const bool on = row < a.rows;
        float x[NV][V], z[NV][V], g[NV][V];
        load_row<T, V, NV>(x, a.x, row * a.x_stride + s.col0, s.lane, a.tg, a.width, on);
        load_row<T, V, NV>(z, a.z, row * a.z_stride + s.col0, s.lane, a.tg, a.width, on);
        load_row<T, V, NV>(g, a.dout, row * a.dout_stride + s.col0, s.lane, a.tg, a.width, on);
        float sq = 0.0f, dot = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float gate = z[j][k] * sigmoid(z[j][k]);
                const float u = a.gate_first ? x[j][k] * gate : x[j][k], e = a.gate_first ? g[j][k] : g[j][k] * gate;
                sq = fmaf(u, u, sq);
                dot = fmaf(e * w[j][k], u, dot);
            }
        sum_group<CTA>(sq, dot, a.tg);
        const float r = rstd_of(sq, a), back = r * r * dot / (float)a.width;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float sg = sigmoid(z[j][k]), gate = z[j][k] * sg;
                const float u = a.gate_first ? x[j][k] * gate : x[j][k], e = a.gate_first ? g[j][k] : g[j][k] * gate;
                const float unit = u * r, du = r * fmaf(e, w[j][k], -u * back);
                dw[j][k] = fmaf(e, unit, dw[j][k]);
                const float dgate = a.gate_first ? du * x[j][k] : g[j][k] * unit * w[j][k];
                x[j][k] = a.gate_first ? du * gate : du;
                z[j][k] = dgate * sg * (1.0f + z[j][k] * (1.0f - sg));
            }
        if (on) {
            store_row<T, V, NV>(a.dx, row * a.dx_stride + s.col0, x, s.lane, a.tg, a.width);
            store_row<T, V, NV>(a.dz, row * a.dz_stride + s.col0, z, s.lane, a.tg, a.width);
        }
    }
    put_parts<V, NV, CTA>(a, s, dw, 0, red);
}

template <typename T, typename R, int NV, bool CTA>
__global__ void __launch_bounds__(CTA ? 512 : kWarpThreads) residual_norm_grad_kernel(const __grid_constant__ NormArgs a) {
    constexpr int V = kVec<T>;
    __shared__ float red[CTA ? 1 : kWarpThreads * NV * V];
    pdl_wait();
    pdl_trigger();
    const Seat<CTA> s(a);
    float w[NV][V], scale[NV][V], dw[NV][V], ds[NV][V];
    load_row<float, V, NV>(w, a.weight, s.col0, s.lane, a.tg, a.width, true);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < V; ++k) {
            dw[j][k] = ds[j][k] = 0.0f;
            scale[j][k] = 1.0f;
        }
    if (a.scale != nullptr) load_row<float, V, NV>(scale, a.scale, s.col0, s.lane, a.tg, a.width, true);
    for (int64_t row0 = (int64_t)blockIdx.x * s.at_once; row0 < a.rows; row0 += (int64_t)gridDim.x * s.at_once) {
        const int64_t row = row0 + s.seat;
        const bool on = row < a.rows;
        float x[NV][V], h[NV][V], g[NV][V], dh[NV][V];
        load_row<T, V, NV>(x, a.x, row * a.x_stride + s.col0, s.lane, a.tg, a.width, on);
        load_row<R, V, NV>(h, a.residual, row * a.residual_stride + s.col0, s.lane, a.tg, a.width, on);
        load_row<T, V, NV>(g, a.dout, row * a.dout_stride + s.col0, s.lane, a.tg, a.width, on);
        load_row<R, V, NV>(dh, a.dres, row * a.dres_stride + s.col0, s.lane, a.tg, a.width, on && a.dres != nullptr);
        float sq = 0.0f, dot = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                h[j][k] = fmaf(scale[j][k], x[j][k], h[j][k]);
                sq = fmaf(h[j][k], h[j][k], sq);
                dot = fmaf(g[j][k] * w[j][k], h[j][k], dot);
            }
        sum_group<CTA>(sq, dot, a.tg);
        const float r = rstd_of(sq, a), back = r * r * dot / (float)a.width;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                dh[j][k] = fmaf(r, fmaf(g[j][k], w[j][k], -h[j][k] * back), dh[j][k]);
                dw[j][k] = fmaf(g[j][k], h[j][k] * r, dw[j][k]);
                ds[j][k] = fmaf(dh[j][k], x[j][k], ds[j][k]);
                x[j][k] = scale[j][k] * dh[j][k];
            }
        if (on) {
            store_row<T, V, NV>(a.dx, row * a.dx_stride + s.col0, x, s.lane, a.tg, a.width);
            store_row<R, V, NV>(a.dresidual, row * a.dresidual_stride + s.col0, dh, s.lane, a.tg, a.width);
        }
    }
    put_parts<V, NV, CTA>(a, s, dw, 0, red);
    if (a.scale != nullptr) put_parts<V, NV, CTA>(a, s, ds, 1, red);
}

// Weight gradients over the CTAs: 32 columns a CTA, eight threads to a column.
constexpr int kJoinThreads = 256, kSlices = kJoinThreads / 32;
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

// CTAs over rows: enough to fill the SMs, no more than there is work.
int rows_grid(const NormArgs& a, const NormCut& c, int groups, int num_sms, bool backward) {
    const int64_t all = (a.rows + c.groups_at_once - 1) / c.groups_at_once;
    const int64_t per_sm = backward ? 2048 / c.threads / 4 : 2048 / c.threads;
    int64_t most = ((int64_t)num_sms * per_sm + groups - 1) / groups;
    if (backward && most > kMaxParts) most = kMaxParts;
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
                                   rows_grid(a, c, groups, ctx->num_sms, false), st));
}
ofrl_status run_backward(const ofrl_norm* ctx, const NormCut& c, const NormArgs& a, bool gated, float* dweight,
                         float* dscale, cudaStream_t st) {
    const int groups = ctx->shape.groups, grid = rows_grid(a, c, groups, ctx->num_sms, true);
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

int64_t norm_bytes(const ofrl_norm_shape& s, int num_sms, bool backward) {
    if (!backward) return 256;
    const NormCut c = norm_cut(s.channels / s.groups, (int)dtype_size(s.dtype));
    NormArgs a;
    std::memset(&a, 0, sizeof(a));
    a.rows = INT32_MAX;
    return 256 + 2 * (int64_t)rows_grid(a, c, s.groups, num_sms, true) * s.channels * 4;
}

}  // namespace
}  // namespace ofrl

using namespace ofrl;

extern "C" {

int64_t ofrl_norm_workspace_bytes(const ofrl_norm_shape* shape, int32_t backward) {
    if (check_shape(shape) != OFRL_OK || (backward != 0 && backward != 1)) return -1;
    int device = 0;
    const int sms = current_sms(&device);
    return norm_bytes(*shape, sms > 0 ? sms : 1, backward != 0);
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
    if (ctx->num_sms > 0) ctx->bytes = norm_bytes(*shape, ctx->num_sms, backward != 0);
    if (ctx->num_sms == 0 || take_memory(&ctx->base, ctx->bytes) != cudaSuccess) {
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
