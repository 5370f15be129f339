// The 2-norm over many tensors, and clipping by it.
//
// The list is cut on the host into segments of at most kSegment elements of
// one tensor; a warp takes every W-th segment, W the launch's warps.  Squares
// are fp32; a lane adds those of one segment into a plain fp32 sum of at most
// kSegment / 32 terms and carries the sums as an unevaluated pair (two-sum),
// so the error does not grow with the number of segments.  The order of every
// addition is fixed by the list alone.
//
// The factor needs every element, so each is read twice.  A list of up to
// kClusterElems elements is one launch of a cluster of eight CTAs, whose sums
// meet in distributed shared memory; a longer one is a launch for the norm
// (its last CTA adds up) and one that scales, from the end of the list, whose
// segments L2 still holds.  Bound by HBM for long lists, by latency for short:
// 150 million elements in 640 tensors, fp32, 92 us for the norm and 191 us for
// the scaling (6.5 and 6.3 TB/s), bf16 52 and 98; 120 thousand elements in 17
// tensors 5.3 us a call, the norm alone 3.5.
// (Hints that keep the list's end in L2 and pass the rest through: 295 us in all
// against 285; streaming stores 286; four or eight CTAs an SM 291.)

#include <cmath>
#include <cstring>
#include <new>

#include "common.cuh"

namespace ofrl {
namespace {

constexpr int kThreads = 256;
constexpr int kSegment = 2048;
constexpr int kMaxList = 1 << 20;
constexpr int kCtasPerSm = 6;
constexpr int kCluster = 8;
constexpr int kClusterThreads = 512;
constexpr int64_t kClusterElems = 1 << 18;

struct Segment {
    uint64_t ptr;
    int32_t count;
    int32_t dtype;
};

struct NormState {
    unsigned int ticket;    // CTAs done; the last one resets it
    float scale;
};

struct NormLaunch {
    const Segment* seg;
    const Segment* out;     // clip: same shape as seg; null: the norm alone
    int64_t n_seg;
    float4* partial;        // [grid]
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

// A sum of squares over lanes: pairs for those from 1 on, times kDown so that
// 2^24 of them do not overflow, and for the ones below, as they are.
struct Sums {
    float s, c, big_s, big_c;
};
constexpr float kDown = 1.0f / (1 << 24), kDownRoot = 1.0f / (1 << 12);

__device__ __forceinline__ Sums sums_of(float s, float c) {
    return s >= 1.0f ? Sums{0.0f, 0.0f, s * kDown, c * kDown} : Sums{s, c, 0.0f, 0.0f};      // a NaN stays below
}
__device__ __forceinline__ void add(Sums& a, const Sums& b) {
    pair_add(a.s, a.c, b.s);
    a.c += b.c;
    pair_add(a.big_s, a.big_c, b.big_s);
    a.big_c += b.big_c;
}
// Once a sum is infinite or NaN, its remainder is NaN and says nothing.
__device__ __forceinline__ float root(const Sums& a) {
    const float low = isfinite(a.s) ? a.s + a.c : a.s, big = isfinite(a.big_s) ? a.big_s + a.big_c : a.big_s;
    return big > 0.0f ? sqrtf(big + low * kDown) / kDownRoot : sqrtf(low);
}
__device__ __forceinline__ Sums warp_sums(Sums a, int from = 16) {
    for (int o = from; o > 0; o >>= 1)
        add(a, {__shfl_down_sync(0xffffffffu, a.s, o), __shfl_down_sync(0xffffffffu, a.c, o),
                __shfl_down_sync(0xffffffffu, a.big_s, o), __shfl_down_sync(0xffffffffu, a.big_c, o)});
    return a;      // lane 0's
}

// Sum over the block; thread 0 has it.
template <int WARPS>
__device__ __forceinline__ Sums block_sums(Sums a) {
    __shared__ Sums part[WARPS];
    a = warp_sums(a);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = a;
    __syncthreads();
    if (threadIdx.x < 32) a = warp_sums(threadIdx.x < WARPS ? part[threadIdx.x] : Sums{0, 0, 0, 0}, WARPS / 2);
    return a;
}

// Elements before the first 16-byte boundary, at most n.
template <typename T>
__device__ __forceinline__ int head_of(uint64_t p, int n) {
    const int h = (int)((16 - (p & 15)) & 15) / (int)sizeof(T);
    return h < n ? h : n;
}
__device__ __forceinline__ float2 halves(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}
__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ float squares(uint64_t ptr, int count) {
    const int lane = threadIdx.x & 31;
    const T* p = reinterpret_cast<const T*>(ptr);
    const int head = head_of<T>(ptr, count);
    constexpr int kVec = 16 / sizeof(T);
    const int vecs = (count - head) / kVec, rest = head + vecs * kVec;
    const uint4* v = reinterpret_cast<const uint4*>(p + head);
    float x = 0.0f;
    auto take = [&](const uint4& u) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                const float e = __uint_as_float(w[i]);
                x = fmaf(e, e, x);
            } else {
                const float2 e = halves(w[i]);
                x = fmaf(e.x, e.x, x);
                x = fmaf(e.y, e.y, x);
            }
        }
    };
    constexpr int kAtOnce = 8;
    int i = lane;
    for (; i + 32 * (kAtOnce - 1) < vecs; i += 32 * kAtOnce) {
        uint4 u[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) u[k] = v[i + 32 * k];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) take(u[k]);
    }
    for (; i < vecs; i += 32) take(v[i]);
    // fewer than kVec elements before and after the vectors
    const int at = lane < head ? lane : rest + lane - head;
    if (lane < head || at < count) {
        const float e = value(p[at]);
        x = fmaf(e, e, x);
    }
    return x;
}

// Squares of this warp's segments.
__device__ __forceinline__ Sums norm_part(const NormLaunch& a, int64_t warp, int64_t warps) {
    float s = 0.0f, c = 0.0f;
    Segment g = {0, 0, 0}, next = {0, 0, 0};
    if (warp < a.n_seg) next = a.seg[warp];
    for (int64_t k = warp; k < a.n_seg; k += warps) {
        g = next;
        if (k + warps < a.n_seg) next = a.seg[k + warps];
        pair_add(s, c, g.dtype == OFRL_DTYPE_F32 ? squares<float>(g.ptr, g.count) : squares<__nv_bfloat16>(g.ptr, g.count));
    }
    return sums_of(s, c);
}

template <typename T>
__device__ __forceinline__ uint4 scaled(uint4 u, float f) {
    uint32_t* x = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
        } else {
            const float2 e = halves(x[i]);
            const __nv_bfloat162 h = __floats2bfloat162_rn(e.x * f, e.y * f);
            x[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    return u;
}

template <typename T>
__device__ __forceinline__ void scale_segment(uint64_t from, uint64_t to, int count, float f) {
    const int lane = threadIdx.x & 31;
    const T* p = reinterpret_cast<const T*>(from);
    T* q = reinterpret_cast<T*>(to);
    auto one = [&](int i) {
        if constexpr (sizeof(T) == 4)
            q[i] = p[i] * f;
        else
            q[i] = __float2bfloat16_rn(value(p[i]) * f);
    };
    if ((from ^ to) & 15) {      // no common boundary: element by element
        for (int i = lane; i < count; i += 32) one(i);
        return;
    }
    const int head = head_of<T>(from, count);
    constexpr int kVec = 16 / sizeof(T);
    const int vecs = (count - head) / kVec, rest = head + vecs * kVec;
    const uint4* v = reinterpret_cast<const uint4*>(p + head);
    uint4* w = reinterpret_cast<uint4*>(q + head);
    constexpr int kAtOnce = 8;
    int i = lane;
    for (; i + 32 * (kAtOnce - 1) < vecs; i += 32 * kAtOnce) {
        uint4 u[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) u[k] = v[i + 32 * k];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) w[i + 32 * k] = scaled<T>(u[k], f);
    }
    for (; i < vecs; i += 32) w[i] = scaled<T>(v[i], f);
    const int at = lane < head ? lane : rest + lane - head;
    if (lane < head || at < count) one(at);
}

// Scales this warp's segments, the last ones first.
__device__ __forceinline__ void scale_part(const NormLaunch& a, int64_t warp, int64_t warps, float f) {
    if (a.out == nullptr || (f == 1.0f && a.out == a.seg) || warp >= a.n_seg) return;
    int64_t k = warp + (a.n_seg - 1 - warp) / warps * warps;
    Segment next = a.seg[k];
    uint64_t next_to = a.out[k].ptr;
    for (; k >= 0; k -= warps) {
        const Segment g = next;
        const uint64_t to = next_to;
        if (k >= warps) {
            next = a.seg[k - warps];
            next_to = a.out[k - warps].ptr;
        }
        if (g.dtype == OFRL_DTYPE_F32)
            scale_segment<float>(g.ptr, to, g.count, f);
        else
            scale_segment<__nv_bfloat16>(g.ptr, to, g.count, f);
    }
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ NormLaunch a) {
    constexpr int W = kThreads / 32;
    pdl_wait();
    const Sums part = block_sums<W>(norm_part(a, blockIdx.x * (int64_t)W + (threadIdx.x >> 5), gridDim.x * (int64_t)W));
    __shared__ bool last;
    if (threadIdx.x == 0) {
        a.partial[blockIdx.x] = make_float4(part.s, part.c, part.big_s, part.big_c);
        __threadfence();
        last = atomicAdd(&a.state->ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (a.out != nullptr) pdl_trigger();      // scale_kernel is next
    if (!last) return;
    __threadfence();
    Sums p = {0, 0, 0, 0};
    for (int b = threadIdx.x; b < gridDim.x; b += kThreads) {
        const float4 x = __ldcg(a.partial + b);
        add(p, {x.x, x.y, x.z, x.w});
    }
    __syncthreads();
    p = block_sums<W>(p);
    if (threadIdx.x == 0) {
        const float norm = root(p);
        a.state->scale = clip_scale(norm, a.max_norm);
        a.state->ticket = 0;
        a.norm_out[0] = norm;
    }
}

__global__ void __launch_bounds__(kThreads) scale_kernel(NormLaunch a) {
    constexpr int W = kThreads / 32;
    pdl_wait();
    scale_part(a, blockIdx.x * (int64_t)W + (threadIdx.x >> 5), gridDim.x * (int64_t)W, a.state->scale);
}

// A segment that stays in registers between its squares and its scaling.
struct Held {
    uint4 u[kSegment * 4 / 16 / 32];
    float edge;      // an element before or after the vectors
};
template <typename T>
__device__ __forceinline__ float hold(uint64_t ptr, int count, Held& h) {
    constexpr int kVec = 16 / sizeof(T), kMine = kSegment / kVec / 32;
    const int lane = threadIdx.x & 31;
    const T* p = reinterpret_cast<const T*>(ptr);
    const int head = head_of<T>(ptr, count), vecs = (count - head) / kVec, rest = head + vecs * kVec;
    const uint4* v = reinterpret_cast<const uint4*>(p + head);
#pragma unroll
    for (int k = 0; k < kMine; ++k) h.u[k] = lane + 32 * k < vecs ? v[lane + 32 * k] : make_uint4(0, 0, 0, 0);
    const int at = lane < head ? lane : rest + lane - head;
    h.edge = lane < head || at < count ? value(p[at]) : 0.0f;
    float x = 0.0f;
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
        const uint32_t w[4] = {h.u[k].x, h.u[k].y, h.u[k].z, h.u[k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                const float e = __uint_as_float(w[i]);
                x = fmaf(e, e, x);
            } else {
                const float2 e = halves(w[i]);
                x = fmaf(e.x, e.x, x);
                x = fmaf(e.y, e.y, x);
            }
        }
    }
    return fmaf(h.edge, h.edge, x);
}
template <typename T>
__device__ __forceinline__ void put_held(uint64_t from, uint64_t to, int count, float f, const Held& h) {
    if ((from ^ to) & 15) return scale_segment<T>(from, to, count, f);
    constexpr int kVec = 16 / sizeof(T), kMine = kSegment / kVec / 32;
    const int lane = threadIdx.x & 31;
    T* q = reinterpret_cast<T*>(to);
    const int head = head_of<T>(from, count), vecs = (count - head) / kVec, rest = head + vecs * kVec;
    uint4* w = reinterpret_cast<uint4*>(q + head);
#pragma unroll
    for (int k = 0; k < kMine; ++k)
        if (lane + 32 * k < vecs) w[lane + 32 * k] = scaled<T>(h.u[k], f);
    const int at = lane < head ? lane : rest + lane - head;
    if (lane < head || at < count) {
        if constexpr (sizeof(T) == 4)
            q[at] = h.edge * f;
        else
            q[at] = __float2bfloat16_rn(h.edge * f);
    }
}

// Both in one cluster.  With a segment for each warp at most, it is read once
// and where it goes to is known before the norm is: 120 thousand elements in 17
// tensors 6.1 us when this was tried, read twice 7.5 (now 5.3).
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kClusterThreads)
norm_cluster_kernel(const __grid_constant__ NormLaunch a) {
    constexpr int W = kClusterThreads / 32;
    __shared__ __align__(16) float4 parts[kCluster];
    const int64_t warp = blockIdx.x * (int64_t)W + (threadIdx.x >> 5), warps = kCluster * (int64_t)W;
    // a CTA's shared memory may be written from outside only once the CTA runs:
    // every CTA says so here and waits for the others before it sends its part
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    pdl_wait();
    const bool once = a.n_seg <= warps;
    Held held;
    Segment g = {0, 0, 0};
    uint64_t to = 0;
    Sums mine_part;
    if (once) {
        if (warp < a.n_seg) {
            g = a.seg[warp];
            if (a.out != nullptr) to = a.out[warp].ptr;
        }
        mine_part = sums_of(g.dtype == OFRL_DTYPE_F32 ? hold<float>(g.ptr, g.count, held)
                                                      : hold<__nv_bfloat16>(g.ptr, g.count, held), 0.0f);
    } else {
        mine_part = norm_part(a, warp, warps);
    }
    const Sums part = block_sums<W>(mine_part);
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (threadIdx.x < 32) {      // this CTA's part to every CTA
        const float s = __shfl_sync(0xffffffffu, part.s, 0), c = __shfl_sync(0xffffffffu, part.c, 0),
                    bs = __shfl_sync(0xffffffffu, part.big_s, 0), bc = __shfl_sync(0xffffffffu, part.big_c, 0);
        if (threadIdx.x < kCluster) {
            uint32_t at;
            const uint32_t mine = static_cast<uint32_t>(__cvta_generic_to_shared(&parts[blockIdx.x]));
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(mine), "r"(threadIdx.x));
            asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(s), "f"(c), "f"(bs), "f"(bc)
                         : "memory");
        }
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    Sums p = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kCluster; ++i) add(p, {parts[i].x, parts[i].y, parts[i].z, parts[i].w});
    const float norm = root(p);
    if (blockIdx.x == 0 && threadIdx.x == 0) a.norm_out[0] = norm;
    const float f = clip_scale(norm, a.max_norm);
    if (!once) return scale_part(a, warp, warps, f);
    if (a.out == nullptr || (f == 1.0f && a.out == a.seg) || warp >= a.n_seg) return;
    if (g.dtype == OFRL_DTYPE_F32)
        put_held<float>(g.ptr, to, g.count, f, held);
    else
        put_held<__nv_bfloat16>(g.ptr, to, g.count, f, held);
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
    int grid;               // 0: one cluster
    void* base;             // the single cudaMalloc
    ofrl::Segment* seg;
    float4* partial;
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

ofrl_status launch(const ofrl_tensors* l, const NormLaunch& a, cudaStream_t st) {
    cudaError_t e;
    if (l->grid == 0) {
        e = launch_pdl(norm_cluster_kernel, dim3(kCluster), dim3(kClusterThreads), 0, st, a);
    } else {
        e = launch_pdl(norm_kernel, dim3(l->grid), dim3(kThreads), 0, st, a);
        if (e == cudaSuccess && a.out != nullptr) e = launch_pdl(scale_kernel, dim3(l->grid), dim3(kThreads), 0, st, a);
    }
    return e == cudaSuccess ? OFRL_OK : OFRL_ECUDA;
}

}  // namespace

extern "C" {

ofrl_status ofrl_tensors_create(const void* const* ptrs, const int64_t* sizes, const int32_t* dtypes, int32_t n,
                                ofrl_tensors** out) {
    if (out == nullptr) return OFRL_EINVAL;
    *out = nullptr;
    if (ptrs == nullptr || sizes == nullptr || dtypes == nullptr || n < 1 || n > kMaxList) return OFRL_EINVAL;
    int64_t n_seg = 0, elems = 0;
    for (int32_t i = 0; i < n; ++i) {
        if (sizes[i] < 0 || sizes[i] > (int64_t)1 << 40) return OFRL_EINVAL;
        if (dtypes[i] != OFRL_DTYPE_F32 && dtypes[i] != OFRL_DTYPE_BF16) return OFRL_EINVAL;
        const uintptr_t p = reinterpret_cast<uintptr_t>(ptrs[i]);
        if (sizes[i] > 0 && (p == 0 || (p & (dtypes[i] == OFRL_DTYPE_F32 ? 3u : 1u)))) return OFRL_EINVAL;
        n_seg += (sizes[i] + kSegment - 1) / kSegment;
        elems += sizes[i];
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
    const int64_t most = (int64_t)l->num_sms * kCtasPerSm, want = (n_seg + kThreads / 32 - 1) / (kThreads / 32);
    l->grid = elems <= kClusterElems ? 0 : (int)(want < most ? want : most);
    const int64_t seg_bytes = (n_seg * (int64_t)sizeof(Segment) + 255) / 256 * 256;
    const int64_t part_bytes = (l->grid * (int64_t)sizeof(float4) + 255) / 256 * 256;
    if (cudaMalloc(&l->base, (size_t)(seg_bytes + part_bytes + 256)) != cudaSuccess) {
        cudaGetLastError();
        delete[] host;
        release(l);
        return OFRL_ECUDA;
    }
    char* b = static_cast<char*>(l->base);
    l->seg = reinterpret_cast<Segment*>(b);
    l->partial = reinterpret_cast<float4*>(b + seg_bytes);
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
    return launch(list, args_of(list, norm_out), static_cast<cudaStream_t>(stream));
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
    return launch(list, a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
