// Selective scan, one token for each environment: states streamed once.

#include "scan.cuh"

namespace ofrl {
namespace scan {
namespace {

constexpr int kStepThreads = 128;

// LS lanes share a channel's state, four floats each; a thread has CPT channels,
// of which it makes one's delta and gate and hands them round.  A CTA keeps its
// channels (decays, biases) over the tokens it takes; the next token's state and
// inputs are on their way while one is worked on, and the state of the third from
// now on its way to L2.  Bound by HBM: 16384 environments, 256 channels of 16
// states, bf16, 570 MB: 102 us, 5.6 TB/s (without L2 asked 107.5; two tokens ahead
// 103.4; three CTAs an SM 109, five, of fewer registers, 116; two channels a thread
// 165).
template <typename T, int LS, int CPT>
__global__ void __launch_bounds__(kStepThreads) scan_step_kernel(const __grid_constant__ StepLaunch a) {
    constexpr int kChannels = kStepThreads / LS * CPT, kOwn = CPT < LS ? CPT : LS;
    static_assert(kOwn == CPT, "each channel has a lane that makes its delta");
    const int d = a.shape.channels, n = a.shape.state_dim, per = d / a.shape.groups;
    const int lane = (int)threadIdx.x % LS, n0 = lane * 4;
    const int ch0 = (int)blockIdx.y * kChannels + (int)threadIdx.x / LS * CPT;      // of CPT, in one group
    const int mine = ch0 + (lane < CPT ? which_channel<LS, CPT>() : 0);
    const bool on = n0 < n && ch0 < d, own = lane < CPT && mine < d;
    const int group = min(ch0, d - 1) / per;
    pdl_wait();
    float4 a2[CPT];
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
        a2[i] = make_float4(0, 0, 0, 0);
        if (on) a2[i] = *reinterpret_cast<const float4*>(a.in.a + (int64_t)(ch0 + i) * n + n0);
        a2[i].x *= kLog2e;
        a2[i].y *= kLog2e;
        a2[i].z *= kLog2e;
        a2[i].w *= kLog2e;
    }
    const float bias = own && a.in.dt_bias != nullptr ? a.in.dt_bias[mine] : 0.0f;
    const float skip = own && a.in.d != nullptr ? a.in.d[mine] : 0.0f;

    struct Token {
        float4 h[CPT];
        Vec<T, 4> b, c;
        T x, dt, z;
        int32_t slot;
    };
    auto fetch = [&](Token& k, int64_t tok, int32_t slot) {
        k.slot = slot;
        if (slot < 0 || slot >= a.slots) return;
        const float* h = a.state_in + ((int64_t)slot * d + ch0) * n + n0;
        const T* bp = static_cast<const T*>(a.in.b) + tok * a.in.b_stride + group * n + n0;
        const T* cp = static_cast<const T*>(a.in.c) + tok * a.in.c_stride + group * n + n0;
        if (on) {
#pragma unroll
            for (int i = 0; i < CPT; ++i) k.h[i] = __ldcs(reinterpret_cast<const float4*>(h + (int64_t)i * n));
            if (a.whole_states) {
                k.b = *reinterpret_cast<const Vec<T, 4>*>(bp);
                k.c = *reinterpret_cast<const Vec<T, 4>*>(cp);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    k.b.v[i] = bp[i];
                    k.c.v[i] = cp[i];
                }
            }
        }
        if (own) {
            k.x = static_cast<const T*>(a.in.x)[tok * a.in.x_stride + mine];
            k.dt = static_cast<const T*>(a.in.dt)[tok * a.in.dt_stride + mine];
            if (a.in.z != nullptr) k.z = static_cast<const T*>(a.in.z)[tok * a.in.z_stride + mine];
        }
    };
    auto slot_of = [&](int64_t tok) {
        return tok >= a.in.tokens ? -1 : a.slot_idx != nullptr ? a.slot_idx[tok] : (int32_t)tok;
    };
    const int64_t step = gridDim.x;
    int64_t tok = blockIdx.x;
    // to L2: a CTA's channels of a slot's state are one piece
    auto ask = [&](int32_t slot) {
        if (threadIdx.x != 0 || slot < 0 || slot >= a.slots) return;
        const int first = (int)blockIdx.y * kChannels;
        prefetch_l2(a.state_in + ((int64_t)slot * d + first) * n, (uint32_t)min(kChannels, d - first) * n * 4);
    };
    Token next;
    fetch(next, tok, slot_of(tok));
    int32_t after = slot_of(tok + step), later = slot_of(tok + 2 * step), further = slot_of(tok + 3 * step);
    for (; tok < a.in.tokens; tok += step) {
        Token k = next;
        if (tok + step < a.in.tokens) fetch(next, tok + step, after);
        ask(further);
        after = later;
        later = further;
        further = slot_of(tok + 4 * step);
        T* out = static_cast<T*>(a.out) + tok * a.out_stride + mine;
        if (k.slot < 0 || k.slot >= a.slots) {
            if (threadIdx.x == 0 && blockIdx.y == 0) atomicAdd(a.status + OFRL_STAT_BAD_INDEX, 1);
            if (own) *out = from_float<T>(0.0f);
            continue;
        }
        float delta = 0.0f, dx = 0.0f;
        if (own) {
            delta = to_float(k.dt) + bias;
            if (a.shape.softplus) delta = softplus(delta);
            dx = delta * to_float(k.x);
        }
        float y[CPT];
        float* h = a.state_out + ((int64_t)k.slot * d + ch0) * n + n0;
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            // the lane that made channel i's delta
            const int from = CPT == 4 ? (i >> 1 & 1) + 2 * (i & 1) : i;
            const float de = __shfl_sync(0xffffffffu, delta, from, LS), u = __shfl_sync(0xffffffffu, dx, from, LS);
            float4& v = k.h[i];
            v.x = fmaf(decay_of(de, a2[i].x), v.x, u * to_float(k.b.v[0]));
            v.y = fmaf(decay_of(de, a2[i].y), v.y, u * to_float(k.b.v[1]));
            v.z = fmaf(decay_of(de, a2[i].z), v.z, u * to_float(k.b.v[2]));
            v.w = fmaf(decay_of(de, a2[i].w), v.w, u * to_float(k.b.v[3]));
            if (on) __stcs(reinterpret_cast<float4*>(h + (int64_t)i * n), v);
            y[i] = on ? to_float(k.c.v[0]) * v.x + to_float(k.c.v[1]) * v.y + to_float(k.c.v[2]) * v.z +
                            to_float(k.c.v[3]) * v.w
                      : 0.0f;
        }
        float sum = sum_states<LS, CPT>(y);
        if (own) {
            if (a.in.d != nullptr) sum = fmaf(skip, to_float(k.x), sum);
            if (a.in.z != nullptr) {
                const float z = to_float(k.z);
                sum *= z * sigmoid(z);
            }
            *out = from_float<T>(sum);
        }
    }
}

template <typename T, int LS, int CPT>
cudaError_t go(const StepLaunch& a, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    constexpr int kChannels = kStepThreads / LS * CPT, kCtasPerSm = 4;
    const int cols = (a.shape.channels + kChannels - 1) / kChannels;
    const int64_t most = ((int64_t)a.num_sms * kCtasPerSm + cols - 1) / cols;
    const int64_t rows = a.in.tokens < most ? a.in.tokens : most;
    const cudaError_t e = opt_in_once(scan_step_kernel<T, LS, CPT>, 0, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(scan_step_kernel<T, LS, CPT>, dim3((unsigned)rows, (unsigned)cols), dim3(kStepThreads), 0, st, a);
}

template <typename T>
cudaError_t run(const StepLaunch& a, cudaStream_t st) {
    switch (lanes_of(a.shape.state_dim)) {
        case 1: return go<T, 1, 1>(a, st);
        case 2: return go<T, 2, 2>(a, st);
        case 4: return go<T, 4, 4>(a, st);
        case 8: return go<T, 8, 4>(a, st);
        default: return go<T, 16, 4>(a, st);
    }
}

}  // namespace

cudaError_t launch_step(const StepLaunch& a, cudaStream_t st) {
    return a.shape.dtype == OFRL_DTYPE_F32 ? run<float>(a, st) : run<__nv_bfloat16>(a, st);
}

}  // namespace scan
}  // namespace ofrl
