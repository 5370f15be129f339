// The 2-norm over many tensors, and clipping by it.
//
// The list is cut on the host into segments of at most kSegment elements of
// one tensor; CTA b takes segments b, b + grid, ...  Squares are fp32; a
// thread adds those of one segment into a plain fp32 sum of at most
// kSegment / kThreads terms and carries the sums as an unevaluated pair
// (two-sum), so the error does not grow with the number of segments.  The
// order of every addition is fixed by the list alone.

#include <cmath>
#include <cstring>
#include <new>

#include "common.cuh"

namespace ofrl {
namespace {

constexpr int kThreads = 256;
constexpr int kSegment = 8192;
constexpr int kMaxList = 1 << 20;
constexpr int kCtasPerSm = 4;

struct Segment {
    uint64_t ptr;
    int32_t count;
    int32_t dtype;
};

struct NormState {
    unsigned int ticket;    // CTAs done; the last one resets it
    float norm, scale;
};

struct NormLaunch {
    const Segment* seg;
    const Segment* out;     // clip: same shape as seg
    int64_t n_seg;
    double* partial;        // [grid]
    NormState* state;
    float max_norm;
    float* norm_out;
};

// s + c holds the running sum: Knuth's two-sum.
__device__ __forceinline__ void pair_add(float& s, float& c, float x) {
    const float t = s + x, z = t - s;
    c += (s - (t - z)) + (x - z);
    s = t;
}

__device__ __forceinline__ double block_sum(double v) {
    __shared__ double warp_part[kThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) warp_part[threadIdx.x >> 5] = v;
    __syncthreads();
    double r = 0.0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) r += warp_part[i];
    __syncthreads();
    return r;
}

__device__ __forceinline__ float load_elem(uint64_t p, int32_t dtype, int i) {
    return dtype == OFRL_DTYPE_F32 ? reinterpret_cast<const float*>(p)[i]
                                   : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ NormLaunch a) {
    float s = 0.0f, c = 0.0f;
    for (int64_t k = blockIdx.x; k < a.n_seg; k += gridDim.x) {
        const Segment g = a.seg[k];
        float x = 0.0f;
        for (int i = threadIdx.x; i < g.count; i += kThreads) {
            const float e = load_elem(g.ptr, g.dtype, i);
            x = fmaf(e, e, x);
        }
        pair_add(s, c, x);
    }
    // once s is infinite or NaN, the remainder c is NaN and says nothing
    const double part = block_sum(isfinite(s) ? (double)s + (double)c : (double)s);
    __shared__ bool last;
    if (threadIdx.x == 0) {
        a.partial[blockIdx.x] = part;
        __threadfence();
        last = atomicAdd(&a.state->ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    double sum = 0.0;
    for (int b = threadIdx.x; b < gridDim.x; b += kThreads) sum += __ldcg(a.partial + b);
    sum = block_sum(sum);
    if (threadIdx.x == 0) {
        const float norm = (float)sqrt(sum);
        a.state->norm = norm;
        a.state->scale = clip_scale(norm, a.max_norm);
        a.state->ticket = 0;
        a.norm_out[0] = norm;
    }
}

__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ NormLaunch a) {
    const float f = a.state->scale;
    for (int64_t k = blockIdx.x; k < a.n_seg; k += gridDim.x) {
        const Segment g = a.seg[k];
        const uint64_t to = a.out[k].ptr;
        if (f == 1.0f && to == g.ptr) continue;
        for (int i = threadIdx.x; i < g.count; i += kThreads) {
            const float e = load_elem(g.ptr, g.dtype, i) * f;
            if (g.dtype == OFRL_DTYPE_F32)
                reinterpret_cast<float*>(to)[i] = e;
            else
                reinterpret_cast<__nv_bfloat16*>(to)[i] = __float2bfloat16_rn(e);
        }
    }
}

}  // namespace
}  // namespace ofrl

struct ofrl_tensors {
    int device;
    int num_sms;
    int32_t n;
    int64_t* sizes;         // host copies: what a clip's two lists must share
    int32_t* dtypes;
    int64_t n_seg;
    int grid;
    void* base;             // the single cudaMalloc
    ofrl::Segment* seg;
    double* partial;
    ofrl::NormState* state;
};

using namespace ofrl;

namespace {

ofrl_status check_list(const ofrl_tensors* l) {
    if (l == nullptr) return OFRL_EINVAL;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return OFRL_ECUDA;
    return dev == l->device ? OFRL_OK : OFRL_EINVAL;
}

void release(ofrl_tensors* l) {
    delete[] l->sizes;
    delete[] l->dtypes;
    delete l;
}

NormLaunch args_of(const ofrl_tensors* l, float* norm_out) {
    NormLaunch a;
    std::memset(&a, 0, sizeof(a));
    a.seg = l->seg;
    a.n_seg = l->n_seg;
    a.partial = l->partial;
    a.state = l->state;
    a.max_norm = INFINITY;
    a.norm_out = norm_out;
    return a;
}

}  // namespace

extern "C" {

ofrl_status ofrl_tensors_create(const void* const* ptrs, const int64_t* sizes, const int32_t* dtypes, int32_t n,
                                ofrl_tensors** out) {
    if (out == nullptr) return OFRL_EINVAL;
    *out = nullptr;
    if (ptrs == nullptr || sizes == nullptr || dtypes == nullptr || n < 1 || n > kMaxList) return OFRL_EINVAL;
    int64_t n_seg = 0;
    for (int32_t i = 0; i < n; ++i) {
        if (sizes[i] < 0 || sizes[i] > (int64_t)1 << 40) return OFRL_EINVAL;
        if (dtypes[i] != OFRL_DTYPE_F32 && dtypes[i] != OFRL_DTYPE_BF16) return OFRL_EINVAL;
        const uintptr_t p = reinterpret_cast<uintptr_t>(ptrs[i]);
        if (sizes[i] > 0 && (p == 0 || (p & (dtypes[i] == OFRL_DTYPE_F32 ? 3u : 1u)))) return OFRL_EINVAL;
        n_seg += (sizes[i] + kSegment - 1) / kSegment;
    }
    ofrl_tensors* l = new (std::nothrow) ofrl_tensors;
    if (l == nullptr) return OFRL_ECUDA;
    std::memset(l, 0, sizeof(*l));
    l->n = n;
    l->n_seg = n_seg;
    l->sizes = new (std::nothrow) int64_t[n];
    l->dtypes = new (std::nothrow) int32_t[n];
    Segment* host = new (std::nothrow) Segment[n_seg > 0 ? n_seg : 1];
    if (l->sizes == nullptr || l->dtypes == nullptr || host == nullptr ||
        cudaGetDevice(&l->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&l->num_sms, cudaDevAttrMultiProcessorCount, l->device) != cudaSuccess) {
        delete[] host;
        release(l);
        return OFRL_ECUDA;
    }
    std::memcpy(l->sizes, sizes, n * sizeof(int64_t));
    std::memcpy(l->dtypes, dtypes, n * sizeof(int32_t));
    int64_t k = 0;
    for (int32_t i = 0; i < n; ++i) {
        const int64_t elem = dtypes[i] == OFRL_DTYPE_F32 ? 4 : 2;
        for (int64_t at = 0; at < sizes[i]; at += kSegment)
            host[k++] = {(uint64_t)reinterpret_cast<uintptr_t>(ptrs[i]) + (uint64_t)(at * elem),
                         (int32_t)(sizes[i] - at < kSegment ? sizes[i] - at : kSegment), dtypes[i]};
    }
    const int64_t most = (int64_t)l->num_sms * kCtasPerSm;
    l->grid = (int)(n_seg < 1 ? 1 : n_seg < most ? n_seg : most);
    const int64_t seg_bytes = (n_seg * (int64_t)sizeof(Segment) + 255) / 256 * 256;
    const int64_t part_bytes = (l->grid * (int64_t)sizeof(double) + 255) / 256 * 256;
    if (cudaMalloc(&l->base, (size_t)(seg_bytes + part_bytes + 256)) != cudaSuccess) {
        cudaGetLastError();
        delete[] host;
        release(l);
        return OFRL_ECUDA;
    }
    char* b = static_cast<char*>(l->base);
    l->seg = reinterpret_cast<Segment*>(b);
    l->partial = reinterpret_cast<double*>(b + seg_bytes);
    l->state = reinterpret_cast<NormState*>(b + seg_bytes + part_bytes);
    const bool ok = cudaMemset(l->state, 0, sizeof(NormState)) == cudaSuccess &&
                    cudaMemcpy(l->seg, host, n_seg * sizeof(Segment), cudaMemcpyHostToDevice) == cudaSuccess &&
                    cudaDeviceSynchronize() == cudaSuccess;
    delete[] host;
    if (!ok) {
        cudaGetLastError();
        cudaFree(l->base);
        release(l);
        return OFRL_ECUDA;
    }
    *out = l;
    return OFRL_OK;
}

ofrl_status ofrl_tensors_destroy(ofrl_tensors* list) {
    if (list == nullptr) return OFRL_OK;
    const cudaError_t e1 = cudaDeviceSynchronize();
    const cudaError_t e2 = cudaFree(list->base);
    release(list);
    return (e1 == cudaSuccess && e2 == cudaSuccess) ? OFRL_OK : OFRL_ECUDA;
}

ofrl_status ofrl_global_norm(ofrl_tensors* list, float* norm_out, void* stream) {
    const ofrl_status s = check_list(list);
    if (s != OFRL_OK) return s;
    if (norm_out == nullptr) return OFRL_EINVAL;
    norm_kernel<<<list->grid, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(args_of(list, norm_out));
    return cudaGetLastError() == cudaSuccess ? OFRL_OK : OFRL_ECUDA;
}

ofrl_status ofrl_global_norm_clip(ofrl_tensors* list, float max_norm, float* norm_out, ofrl_tensors* out,
                                  void* stream) {
    ofrl_status s = check_list(list);
    if (s == OFRL_OK && out != nullptr) s = check_list(out);
    if (s != OFRL_OK) return s;
    if (norm_out == nullptr || !(max_norm > 0.0f)) return OFRL_EINVAL;   // also rejects NaN
    if (out != nullptr && out != list &&
        (out->n != list->n || std::memcmp(out->sizes, list->sizes, list->n * sizeof(int64_t)) != 0 ||
         std::memcmp(out->dtypes, list->dtypes, list->n * sizeof(int32_t)) != 0))
        return OFRL_EINVAL;
    NormLaunch a = args_of(list, norm_out);
    a.max_norm = max_norm;
    a.out = out != nullptr ? out->seg : list->seg;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    norm_kernel<<<list->grid, kThreads, 0, st>>>(a);
    scale_kernel<<<list->grid, kThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? OFRL_OK : OFRL_ECUDA;
}

}  // extern "C"
