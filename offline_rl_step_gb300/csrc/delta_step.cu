// One token per environment: the recurrence itself, states streamed once.

#include "delta.cuh"

namespace ofrl {
namespace delta {
namespace {

constexpr int kStepThreads = 128;
constexpr int kStepRows = 16;      // state rows (value channels) per CTA

// One CTA: kStepRows rows of one (token, value head) state.  A row of k_dim
// floats lies across LANES lanes, four floats each; both dot products of a
// row (with k and with q) come from one read of it:
//   o = scale (a S q + u (k q)),  u = beta (v - a S k),  S' = a S + u k^T.
template <typename T, int LANES>
__global__ void __launch_bounds__(kStepThreads) delta_step_kernel(const __grid_constant__ StepLaunch a) {
    const int dk = a.shape.k_dim, dv = a.shape.v_dim, hv = a.shape.v_heads;
    const int slices = (dv + kStepRows - 1) / kStepRows;
    const int64_t item = blockIdx.x / slices;
    const int slice = blockIdx.x % slices;
    const int64_t tok = item / hv;
    const int head = (int)(item % hv), khead = head / (hv / a.shape.k_heads);
    const T* vp = static_cast<const T*>(a.in.v) + tok * a.in.v_stride + (int64_t)head * dv;
    T* op = static_cast<T*>(a.out) + (tok * hv + head) * dv;
    const int row_end = min(dv, (slice + 1) * kStepRows);
    const int32_t slot = a.slot_idx ? a.slot_idx[tok] : (int32_t)tok;
    if (slot < 0 || slot >= a.slots) {
        if (threadIdx.x == 0 && head == 0 && slice == 0) atomicAdd(a.status + OFRL_STAT_BAD_INDEX, 1);
        for (int r = slice * kStepRows + threadIdx.x; r < row_end; r += kStepThreads) op[r] = from_f<T>(0.0f);
        return;
    }
    const int lane = threadIdx.x % LANES, c = lane * 4;
    const bool on = c < dk;
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
    auto row_sum = [](float x) {
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        return x;
    };
    const float kq = row_sum(kx[0] * qx[0] + kx[1] * qx[1] + kx[2] * qx[2] + kx[3] * qx[3]);
    const float decay = expf(to_f(static_cast<const T*>(a.in.g)[tok * a.in.g_stride + head]));
    const float beta = to_f(static_cast<const T*>(a.in.beta)[tok * a.in.beta_stride + head]);
    const int64_t base = ((int64_t)slot * hv + head) * dv * dk;
    constexpr int kRowsAtOnce = kStepThreads / LANES;
    for (int r0 = slice * kStepRows; r0 < row_end; r0 += kRowsAtOnce) {   // every lane takes every turn (shuffles)
        const int r = r0 + threadIdx.x / LANES;
        const bool live = r < row_end;
        float4 s = make_float4(0, 0, 0, 0);
        if (live && on) s = *reinterpret_cast<const float4*>(a.state_in + base + (int64_t)r * dk + c);
        const float sk = row_sum(s.x * kx[0] + s.y * kx[1] + s.z * kx[2] + s.w * kx[3]);
        const float sq = row_sum(s.x * qx[0] + s.y * qx[1] + s.z * qx[2] + s.w * qx[3]);
        if (!live) continue;
        const float u = beta * (to_f(vp[r]) - decay * sk);
        if (on) {
            s.x = decay * s.x + u * kx[0];
            s.y = decay * s.y + u * kx[1];
            s.z = decay * s.z + u * kx[2];
            s.w = decay * s.w + u * kx[3];
            *reinterpret_cast<float4*>(a.state_out + base + (int64_t)r * dk + c) = s;
        }
        if (lane == 0) op[r] = from_f<T>(a.in.scale * (decay * sq + u * kq));
    }
}

template <typename T>
cudaError_t run_step(const StepLaunch& a, cudaStream_t st) {
    const int slices = (a.shape.v_dim + kStepRows - 1) / kStepRows;
    const int64_t grid = a.in.tokens * a.shape.v_heads * slices;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    if (a.shape.k_dim > 64)
        delta_step_kernel<T, 32><<<(unsigned)grid, kStepThreads, 0, st>>>(a);
    else if (a.shape.k_dim > 32)
        delta_step_kernel<T, 16><<<(unsigned)grid, kStepThreads, 0, st>>>(a);
    else
        delta_step_kernel<T, 8><<<(unsigned)grid, kStepThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_step(const StepLaunch& a, cudaStream_t st) {
    return a.shape.dtype == OFRL_DTYPE_F32 ? run_step<float>(a, st) : run_step<__nv_bfloat16>(a, st);
}

}  // namespace delta
}  // namespace ofrl
