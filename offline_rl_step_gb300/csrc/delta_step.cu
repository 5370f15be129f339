// One token per environment: the recurrence itself, states streamed once.

#include <type_traits>

#include "delta.cuh"

namespace ofrl {
namespace delta {
namespace {

constexpr int kAtOnce = 4;         // rows of one lane group, all in flight at once

// One CTA: kAtOnce rows per lane group of one (token, value head) state.  A
// row of k_dim floats lies across LANES lanes, four floats each; both dot
// products of a row (with k and with q) come from one read of it:
//   o = scale (a S q + u (k q)),  u = beta (v - a S k),  S' = a S + u k^T.
// Bound by HBM: every state element is read and written once.  300 tokens, eight
// heads of 128 x 128: 53 us, 6.0 TB/s; 16384 tokens, two of 64 x 64, fp32: 177
// us, 6.2 TB/s; one token 2.8 us, a launch's latency.
template <int LANES>
constexpr int step_rows() { return kStepThreads / LANES * kAtOnce; }

template <typename T, int LANES>
__global__ void __launch_bounds__(kStepThreads) delta_step_kernel(const __grid_constant__ StepLaunch a) {
    pdl_wait();
    const int dk = a.shape.k_dim, dv = a.shape.v_dim, hv = a.shape.v_heads;
    constexpr int kRows = step_rows<LANES>();
    const unsigned slices = (unsigned)(dv + kRows - 1) / kRows;
    const unsigned item = blockIdx.x / slices;
    const int row0 = (int)(blockIdx.x - item * slices) * kRows;
    const int64_t tok = item / (unsigned)hv;
    const int head = (int)(item % (unsigned)hv), khead = head / (hv / a.shape.k_heads);
    const int lane = threadIdx.x % LANES, c = lane * 4;
    const bool on = c < dk;
    const int32_t slot = a.slot_idx ? a.slot_idx[tok] : (int32_t)tok;
    T* op = static_cast<T*>(a.out) + (tok * hv + head) * dv;
    if (slot < 0 || slot >= a.slots) {
        if (threadIdx.x == 0 && head == 0 && row0 == 0) atomicAdd(a.status + OFRL_STAT_BAD_INDEX, 1);
        for (int r = row0 + threadIdx.x; r < min(dv, row0 + kRows); r += kStepThreads) op[r] = from_f<T>(0.0f);
        return;
    }
    const int64_t base = ((int64_t)slot * hv + head) * dv * dk;
    float4 s[kAtOnce];
    int row[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
        row[i] = row0 + (int)threadIdx.x / LANES + i * (kStepThreads / LANES);
        s[i] = make_float4(0, 0, 0, 0);
        if (on && row[i] < dv) s[i] = __ldcs(reinterpret_cast<const float4*>(a.state_in + base + (int64_t)row[i] * dk + c));
    }
    float kx[4] = {0, 0, 0, 0}, qx[4] = {0, 0, 0, 0};
    if (on) {
        const T* kp = static_cast<const T*>(a.in.k) + tok * a.in.k_stride + (int64_t)khead * dk + c;
        const T* qp = static_cast<const T*>(a.in.q) + tok * a.in.q_stride + (int64_t)khead * dk + c;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            kx[i] = to_f(kp[i]);
            qx[i] = to_f(qp[i]);
        }
    }
    const T* vp = static_cast<const T*>(a.in.v) + tok * a.in.v_stride + (int64_t)head * dv;
    float v[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) v[i] = row[i] < dv ? to_f(vp[row[i]]) : 0.0f;
    const float decay = expf(to_f(static_cast<const T*>(a.in.g)[tok * a.in.g_stride + head]));
    const float beta = to_f(static_cast<const T*>(a.in.beta)[tok * a.in.beta_stride + head]);
    auto row_sum = [](float x) {
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        return x;
    };
    const float kq = row_sum(kx[0] * qx[0] + kx[1] * qx[1] + kx[2] * qx[2] + kx[3] * qx[3]);
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
        const float sk = row_sum(s[i].x * kx[0] + s[i].y * kx[1] + s[i].z * kx[2] + s[i].w * kx[3]);
        const float sq = row_sum(s[i].x * qx[0] + s[i].y * qx[1] + s[i].z * qx[2] + s[i].w * qx[3]);
        const float u = beta * (v[i] - decay * sk);
        if (row[i] >= dv) continue;
        if (on) {
            s[i].x = decay * s[i].x + u * kx[0];
            s[i].y = decay * s[i].y + u * kx[1];
            s[i].z = decay * s[i].z + u * kx[2];
            s[i].w = decay * s[i].w + u * kx[3];
            __stcs(reinterpret_cast<float4*>(a.state_out + base + (int64_t)row[i] * dk + c), s[i]);
        }
        if (lane == 0) op[row[i]] = from_f<T>(a.in.scale * (decay * sq + u * kq));
    }
}

template <typename T, int LANES>
cudaError_t go(const StepLaunch& a, cudaStream_t st) {
    const int rows = step_rows<LANES>(), slices = (a.shape.v_dim + rows - 1) / rows;
    const int64_t grid = a.in.tokens * a.shape.v_heads * slices;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    return launch_pdl(delta_step_kernel<T, LANES>, dim3((unsigned)grid), dim3(kStepThreads), 0, st, a);
}

template <typename T>
cudaError_t run_step(const StepLaunch& a, cudaStream_t st) {
    if (a.shape.k_dim > 64) return go<T, 32>(a, st);
    return a.shape.k_dim > 32 ? go<T, 16>(a, st) : go<T, 8>(a, st);
}

// Short episodes, token by token: the same recurrence with the state in
// registers.  A lane group has kRecurRows rows; a token costs two dot products
// over the group's lanes and the update, about 0.28 us in all, so
// episodes of a few dozen tokens are through before the chunked path's two
// launches would be (16 episodes of 16 tokens, two heads of 64, fp32: 7.0 us
// against 13.8).  What bounds it is that step's latency; with many episodes the
// shuffles of its dot products, 0.11 ns for 32 lanes' share of a token.  Tokens are loaded kAhead at a time, a round ahead.
constexpr int kAhead = 4;

template <typename T, int LANES>
__global__ void __launch_bounds__(kStepThreads) delta_recur_kernel(const __grid_constant__ SeqLaunch a) {
    pdl_wait();
    const int dk = a.shape.k_dim, dv = a.shape.v_dim, hv = a.shape.v_heads;
    constexpr int kRows = recur_rows(LANES), kGroups = kStepThreads / LANES;
    const unsigned slices = (unsigned)(dv + kRows - 1) / kRows;
    const unsigned item = blockIdx.x / slices;
    const int row0 = (int)(blockIdx.x - item * slices) * kRows + (int)threadIdx.x / LANES;
    const int e = (int)(item / (unsigned)hv), head = (int)(item % (unsigned)hv), khead = head / (hv / a.shape.k_heads);
    const int lane = threadIdx.x % LANES, c = lane * 4;
    const bool on = c < dk;
    const int32_t tokens = (int32_t)a.in.tokens;
    const Span sp = span_of(a.ends, e, tokens);
    if (threadIdx.x == 0 && head == 0 && blockIdx.x == item * slices && span_bad(a.ends, e, tokens))
        atomicAdd(a.status + OFRL_STAT_BAD_INDEX, 1);
    const T* kp = static_cast<const T*>(a.in.k) + (int64_t)sp.start * a.in.k_stride + (int64_t)khead * dk + (on ? c : 0);
    const T* qp = static_cast<const T*>(a.in.q) + (int64_t)sp.start * a.in.q_stride + (int64_t)khead * dk + (on ? c : 0);
    const T* vp = static_cast<const T*>(a.in.v) + (int64_t)sp.start * a.in.v_stride + (int64_t)head * dv;
    const T* gp = static_cast<const T*>(a.in.g) + (int64_t)sp.start * a.in.g_stride + head;
    const T* bp = static_cast<const T*>(a.in.beta) + (int64_t)sp.start * a.in.beta_stride + head;
    T* op = static_cast<T*>(a.out) + ((int64_t)sp.start * hv + head) * dv;
    struct Token {
        T k[4], q[4], v[kRecurRows], g, b;
    };
    auto load = [&](Token (&x)[kAhead], int t0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int64_t t = min(t0 + i, sp.len - 1);
            using Four = typename std::conditional<sizeof(T) == 4, uint4, uint2>::type;
            *reinterpret_cast<Four*>(x[i].k) = *reinterpret_cast<const Four*>(kp + t * a.in.k_stride);
            *reinterpret_cast<Four*>(x[i].q) = *reinterpret_cast<const Four*>(qp + t * a.in.q_stride);
#pragma unroll
            for (int r = 0; r < kRecurRows; ++r) x[i].v[r] = vp[t * a.in.v_stride + min(row0 + r * kGroups, dv - 1)];
            x[i].g = gp[t * a.in.g_stride];
            x[i].b = bp[t * a.in.beta_stride];
        }
    };
    const int64_t base = ((int64_t)e * hv + head) * dv * dk;
    float s[kRecurRows][4];
#pragma unroll
    for (int r = 0; r < kRecurRows; ++r) {
        float4 x = make_float4(0, 0, 0, 0);
        const int row = row0 + r * kGroups;
        if (a.init && on && row < dv) x = *reinterpret_cast<const float4*>(a.init + base + (int64_t)row * dk + c);
        s[r][0] = x.x;
        s[r][1] = x.y;
        s[r][2] = x.z;
        s[r][3] = x.w;
    }
    auto row_sum = [](float x) {
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        return x;
    };
    Token now[kAhead], next[kAhead];
    if (sp.len > 0) load(now, 0);
    for (int t0 = 0; t0 < sp.len; t0 += kAhead) {
        load(next, t0 + kAhead);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (t0 + i < sp.len) {      // the same for every lane
                float k[4], q[4];
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    k[z] = on ? to_f(now[i].k[z]) : 0.0f;
                    q[z] = on ? to_f(now[i].q[z]) : 0.0f;
                }
                const float decay = expf(to_f(now[i].g)), beta = to_f(now[i].b);
                const float kq = row_sum(k[0] * q[0] + k[1] * q[1] + k[2] * q[2] + k[3] * q[3]);
#pragma unroll
                for (int r = 0; r < kRecurRows; ++r) {
                    const float sk = row_sum(s[r][0] * k[0] + s[r][1] * k[1] + s[r][2] * k[2] + s[r][3] * k[3]);
                    const float sq = row_sum(s[r][0] * q[0] + s[r][1] * q[1] + s[r][2] * q[2] + s[r][3] * q[3]);
                    const float u = beta * (to_f(now[i].v[r]) - decay * sk);
#pragma unroll
                    for (int z = 0; z < 4; ++z) s[r][z] = decay * s[r][z] + u * k[z];
                    const int row = row0 + r * kGroups;
                    if (lane == 0 && row < dv)
                        op[(int64_t)(t0 + i) * hv * dv + row] = from_f<T>(a.in.scale * (decay * sq + u * kq));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) now[i] = next[i];
    }
    if (a.final_state)
#pragma unroll
        for (int r = 0; r < kRecurRows; ++r) {
            const int row = row0 + r * kGroups;
            if (on && row < dv)
                *reinterpret_cast<float4*>(a.final_state + base + (int64_t)row * dk + c) =
                    make_float4(s[r][0], s[r][1], s[r][2], s[r][3]);
        }
}

template <typename T, int LANES>
cudaError_t go_recur(const SeqLaunch& a, cudaStream_t st) {
    const int rows = recur_rows(LANES), slices = (a.shape.v_dim + rows - 1) / rows;
    const int64_t grid = (int64_t)a.episodes * a.shape.v_heads * slices;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    return launch_pdl(delta_recur_kernel<T, LANES>, dim3((unsigned)grid), dim3(kStepThreads), 0, st, a);
}

template <typename T>
cudaError_t run_recur(const SeqLaunch& a, cudaStream_t st) {
    if (a.shape.k_dim > 64) return go_recur<T, 32>(a, st);
    return a.shape.k_dim > 32 ? go_recur<T, 16>(a, st) : go_recur<T, 8>(a, st);
}

}  // namespace

cudaError_t launch_step(const StepLaunch& a, cudaStream_t st) {
    return a.shape.dtype == OFRL_DTYPE_F32 ? run_step<float>(a, st) : run_step<__nv_bfloat16>(a, st);
}

cudaError_t launch_recur(const SeqLaunch& a, cudaStream_t st) {
    return a.shape.dtype == OFRL_DTYPE_F32 ? run_recur<float>(a, st) : run_recur<__nv_bfloat16>(a, st);
}

}  // namespace delta
}  // namespace ofrl
