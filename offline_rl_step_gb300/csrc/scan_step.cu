// Selective scan, one token for each environment: states streamed once.

#include "scan.cuh"

namespace ofrl {
namespace scan {
namespace {

constexpr int kAtOnce = 4;         // channels of a lane group, all in flight
constexpr int kStepThreads = 128;

// LS lanes have a channel's state, four floats each; a lane group has kAtOnce
// channels, which share what it loads of B and C.
template <typename T, int LS>
__global__ void __launch_bounds__(kStepThreads) scan_step_kernel(const __grid_constant__ StepLaunch a) {
    pdl_wait();
    pdl_trigger();
    constexpr int kGroups = kStepThreads / LS, kChannels = kGroups * kAtOnce;
    const int d = a.shape.channels, n = a.shape.state_dim, per = d / a.shape.groups;
    const unsigned slices = (unsigned)(d + kChannels - 1) / kChannels;
    const int64_t tok = blockIdx.x / slices;
    const int ch0 = (int)(blockIdx.x % slices) * kChannels + (int)threadIdx.x / LS;
    const int n0 = (int)threadIdx.x % LS * 4;
    const bool on = n0 < n;
    const int32_t slot = a.slot_idx ? a.slot_idx[tok] : (int32_t)tok;
    T* out = static_cast<T*>(a.out) + tok * a.out_stride;
    if (slot < 0 || slot >= a.slots) {
        if (threadIdx.x == 0 && blockIdx.x % slices == 0) atomicAdd(a.status + OFRL_STAT_BAD_INDEX, 1);
        if (threadIdx.x % LS == 0)
            for (int i = 0; i < kAtOnce; ++i)
                if (ch0 + i * kGroups < d) out[ch0 + i * kGroups] = from_float<T>(0.0f);
        return;
    }
    const int64_t base = (int64_t)slot * d * n + n0;
    float4 h[kAtOnce], a2[kAtOnce];
    float x[kAtOnce], dt[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
        const int ch = ch0 + i * kGroups;
        h[i] = a2[i] = make_float4(0, 0, 0, 0);
        x[i] = dt[i] = 0.0f;
        if (ch >= d) continue;
        if (on) h[i] = __ldcs(reinterpret_cast<const float4*>(a.state_in + base + (int64_t)ch * n));
        if (on) a2[i] = *reinterpret_cast<const float4*>(a.in.a + (int64_t)ch * n + n0);
        x[i] = to_float(static_cast<const T*>(a.in.x)[tok * a.in.x_stride + ch]);
        dt[i] = to_float(static_cast<const T*>(a.in.dt)[tok * a.in.dt_stride + ch]);
    }
    int group = -1;
    float b[4], c[4];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
        const int ch = ch0 + i * kGroups;
        if (ch < d && ch / per != group) {
            group = ch / per;
            const T* bp = static_cast<const T*>(a.in.b) + tok * a.in.b_stride + group * n + n0;
            const T* cp = static_cast<const T*>(a.in.c) + tok * a.in.c_stride + group * n + n0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                b[k] = on ? to_float(bp[k]) : 0.0f;
                c[k] = on ? to_float(cp[k]) : 0.0f;
            }
        }
        float y = 0.0f;
        if (ch < d && on) {
            const float delta = delta_of(dt[i], a.in.dt_bias != nullptr ? a.in.dt_bias[ch] : 0.0f, a.shape.softplus);
            const float dx = delta * x[i], l = delta * kLog2e;
            h[i].x = fmaf(exp2_of(l * a2[i].x), h[i].x, dx * b[0]);
            h[i].y = fmaf(exp2_of(l * a2[i].y), h[i].y, dx * b[1]);
            h[i].z = fmaf(exp2_of(l * a2[i].z), h[i].z, dx * b[2]);
            h[i].w = fmaf(exp2_of(l * a2[i].w), h[i].w, dx * b[3]);
            __stcs(reinterpret_cast<float4*>(a.state_out + base + (int64_t)ch * n), h[i]);
            y = c[0] * h[i].x + c[1] * h[i].y + c[2] * h[i].z + c[3] * h[i].w;
        }
#pragma unroll
        for (int o = LS / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        if (ch < d && n0 == 0) {
            if (a.in.d != nullptr) y = fmaf(a.in.d[ch], x[i], y);
            if (a.in.z != nullptr) {
                const float z = to_float(static_cast<const T*>(a.in.z)[tok * a.in.z_stride + ch]);
                y *= z * sigmoid(z);
            }
            out[ch] = from_float<T>(y);
        }
    }
}

template <typename T, int LS>
cudaError_t go(const StepLaunch& a, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    const int channels = kStepThreads / LS * kAtOnce;
    const int64_t grid = a.in.tokens * ((a.shape.channels + channels - 1) / channels);
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    const cudaError_t e = opt_in_once(scan_step_kernel<T, LS>, 0, done);
    return e != cudaSuccess ? e : launch_pdl(scan_step_kernel<T, LS>, dim3((unsigned)grid), dim3(kStepThreads), 0, st, a);
}

template <typename T>
cudaError_t run(const StepLaunch& a, cudaStream_t st) {
    switch (lanes_of(a.shape.state_dim)) {
        case 1: return go<T, 1>(a, st);
        case 2: return go<T, 2>(a, st);
        case 4: return go<T, 4>(a, st);
        case 8: return go<T, 8>(a, st);
        default: return go<T, 16>(a, st);
    }
}

}  // namespace

cudaError_t launch_step(const StepLaunch& a, cudaStream_t st) {
    return a.shape.dtype == OFRL_DTYPE_F32 ? run<float>(a, st) : run<__nv_bfloat16>(a, st);
}

}  // namespace scan
}  // namespace ofrl
