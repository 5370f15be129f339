// C entry points of the sequence memory: argument checks, the context and
// the launches.  Nothing here allocates except ofrl_delta_create.

#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>

#include "delta.cuh"

using namespace ofrl;
using namespace ofrl::delta;

namespace {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
inline ofrl_status cuda_status(cudaError_t e) { return e == cudaSuccess ? OFRL_OK : OFRL_ECUDA; }

ofrl_status check_shape(const ofrl_delta_shape* s) {
    if (s == nullptr) return OFRL_EINVAL;
    if (s->k_heads < 1 || s->v_heads < 1 || s->v_heads > 1024 || s->v_heads % s->k_heads != 0) return OFRL_EINVAL;
    if (s->k_dim < 1 || s->v_dim < 1) return OFRL_EINVAL;
    if (s->dtype != OFRL_DTYPE_F32 && s->dtype != OFRL_DTYPE_BF16) return OFRL_EINVAL;
    if (s->k_dim > kMaxDim || s->v_dim > kMaxDim || (s->k_dim & 7) || (s->v_dim & 7)) return OFRL_EUNSUPPORTED;
    return OFRL_OK;
}

bool counts_ok(int64_t tokens, int64_t episodes) {
    return tokens >= 0 && tokens <= INT32_MAX && episodes >= 0 && episodes <= INT32_MAX;
}

int64_t elem_size(const ofrl_delta_shape& s) { return s.dtype == OFRL_DTYPE_F32 ? 4 : 2; }
int64_t states_bytes(const ofrl_delta_shape& s, int64_t count) { return count * s.v_heads * s.v_dim * s.k_dim * 4; }

struct Layout {
    int64_t off_status, off_counter, off_scratch, off_parts, total;
};

Layout layout_of(const ofrl_delta_shape& s, int64_t max_tokens, int64_t max_episodes, bool backward, int num_sms) {
    Layout L;
    int64_t o = 0;
    auto take = [&](int64_t bytes) { const int64_t at = o; o = round_up(o + bytes, 256); return at; };
    L.off_status = take((int64_t)OFRL_STAT_WORDS * 4);
    L.off_counter = take(4);
    L.off_scratch = take(scratch_bytes(s, max_tokens, max_episodes, backward));
    L.off_parts = take(parts_bytes(s, max_tokens, num_sms));
    L.total = o;
    return L;
}

int sm_count(int* device) {
    int sms = 0;
    if (cudaGetDevice(device) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, *device) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return sms;
}

ofrl_status check_ctx(const ofrl_delta* ctx) {
    if (ctx == nullptr) return OFRL_EINVAL;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return OFRL_ECUDA;
    return dev == ctx->device ? OFRL_OK : OFRL_EINVAL;
}

// A token buffer's stride: at least its width, 16-byte rows, and (stride *
// tokens) addressable.
bool stride_ok(int64_t stride, int64_t width, int64_t elem, bool rows16) {
    if (stride < width || stride > (int64_t)1 << 40) return false;
    return !rows16 || (stride * elem) % 16 == 0;
}

ofrl_status check_tokens(const ofrl_delta* ctx, const ofrl_delta_tokens* t) {
    if (t == nullptr) return OFRL_EINVAL;
    if (t->tokens < 0 || t->tokens > INT32_MAX || !std::isfinite(t->scale)) return OFRL_EINVAL;
    if (t->tokens == 0) return OFRL_OK;
    const ofrl_delta_shape& s = ctx->shape;
    const int64_t e = elem_size(s), qk = (int64_t)s.k_heads * s.k_dim, vv = (int64_t)s.v_heads * s.v_dim;
    if (!t->q || !t->k || !t->v || !t->g || !t->beta) return OFRL_EINVAL;
    if (!aligned16(t->q) || !aligned16(t->k) || !aligned16(t->v)) return OFRL_EINVAL;
    if ((reinterpret_cast<uintptr_t>(t->g) | reinterpret_cast<uintptr_t>(t->beta)) & (uintptr_t)(e - 1))
        return OFRL_EINVAL;
    if (!stride_ok(t->q_stride, qk, e, true) || !stride_ok(t->k_stride, qk, e, true) ||
        !stride_ok(t->v_stride, vv, e, true) || !stride_ok(t->g_stride, s.v_heads, e, false) ||
        !stride_ok(t->beta_stride, s.v_heads, e, false))
        return OFRL_EINVAL;
    return OFRL_OK;
}

ofrl_status check_sequence(const ofrl_delta* ctx, const ofrl_delta_tokens* in, const int32_t* ends, int32_t episodes) {
    ofrl_status s = check_ctx(ctx);
    if (s == OFRL_OK) s = check_tokens(ctx, in);
    if (s != OFRL_OK) return s;
    if (episodes < 0 || (episodes > 0 && ends == nullptr)) return OFRL_EINVAL;
    if (in->tokens > 0 && episodes == 0) return OFRL_EINVAL;
    if (in->tokens > ctx->max_tokens || episodes > ctx->max_episodes) return OFRL_EINVAL;
    return OFRL_OK;
}

SeqLaunch base_launch(const ofrl_delta* ctx, const ofrl_delta_tokens* in, const int32_t* ends, int32_t episodes) {
    SeqLaunch a;
    std::memset(&a, 0, sizeof(a));
    a.shape = ctx->shape;
    a.in = *in;
    a.ends = ends;
    a.episodes = episodes;
    a.scratch = ctx->scratch;
    a.parts = ctx->parts;
    a.counter = ctx->counter;
    a.status = ctx->status;
    a.num_sms = ctx->num_sms;
    return a;
}

}  // namespace

extern "C" {

int64_t ofrl_delta_workspace_bytes(const ofrl_delta_shape* shape, int64_t max_tokens, int32_t max_episodes,
                                   int32_t backward) {
    if (check_shape(shape) != OFRL_OK || !counts_ok(max_tokens, max_episodes) || (backward != 0 && backward != 1))
        return -1;
    int device = 0;
    return layout_of(*shape, max_tokens, max_episodes, backward != 0, sm_count(&device)).total;
}

int64_t ofrl_delta_saved_bytes(const ofrl_delta_shape* shape, int64_t tokens, int32_t num_episodes) {
    if (check_shape(shape) != OFRL_OK || !counts_ok(tokens, num_episodes)) return -1;
    return saved_bytes(*shape, tokens, num_episodes);
}

ofrl_status ofrl_delta_create(const ofrl_delta_shape* shape, int64_t max_tokens, int32_t max_episodes,
                              int32_t backward, ofrl_delta** out) {
    if (out == nullptr) return OFRL_EINVAL;
    *out = nullptr;
    const ofrl_status s = check_shape(shape);
    if (s != OFRL_OK) return s;
    if (!counts_ok(max_tokens, max_episodes) || (backward != 0 && backward != 1)) return OFRL_EINVAL;
    ofrl_delta* ctx = new (std::nothrow) ofrl_delta;
    if (ctx == nullptr) return OFRL_ECUDA;
    std::memset(ctx, 0, sizeof(*ctx));
    ctx->num_sms = sm_count(&ctx->device);
    if (ctx->num_sms == 0) {
        delete ctx;
        return OFRL_ECUDA;
    }
    const Layout L = layout_of(*shape, max_tokens, max_episodes, backward != 0, ctx->num_sms);
    ctx->shape = *shape;
    ctx->max_tokens = max_tokens;
    ctx->max_episodes = max_episodes;
    ctx->backward = backward;
    ctx->bytes = L.total;
    if (cudaMalloc(&ctx->base, (size_t)L.total) != cudaSuccess) {
        cudaGetLastError();
        delete ctx;
        return OFRL_ECUDA;
    }
    char* b = static_cast<char*>(ctx->base);
    ctx->status = reinterpret_cast<int32_t*>(b + L.off_status);
    ctx->counter = reinterpret_cast<unsigned*>(b + L.off_counter);
    ctx->scratch = reinterpret_cast<uint8_t*>(b + L.off_scratch);
    ctx->parts = reinterpret_cast<uint8_t*>(b + L.off_parts);
    if (cudaMemset(ctx->status, 0, OFRL_STAT_WORDS * 4) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) {
        cudaFree(ctx->base);
        delete ctx;
        return OFRL_ECUDA;
    }
    *out = ctx;
    return OFRL_OK;
}

ofrl_status ofrl_delta_destroy(ofrl_delta* ctx) {
    if (ctx == nullptr) return OFRL_OK;
    const cudaError_t e1 = cudaDeviceSynchronize();
    const cudaError_t e2 = cudaFree(ctx->base);
    delete ctx;
    return (e1 == cudaSuccess && e2 == cudaSuccess) ? OFRL_OK : OFRL_ECUDA;
}

ofrl_status ofrl_delta_poll_status(ofrl_delta* ctx, void* stream, int32_t* words_out) {
    const ofrl_status s = check_ctx(ctx);
    if (s != OFRL_OK) return s;
    if (words_out == nullptr) return OFRL_EINVAL;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemcpyAsync(words_out, ctx->status, OFRL_STAT_WORDS * 4, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaMemsetAsync(ctx->status, 0, OFRL_STAT_WORDS * 4, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    return cuda_status(e);
}

ofrl_status ofrl_delta_forward(ofrl_delta* ctx, const ofrl_delta_tokens* in, const int32_t* episode_ends,
                               int32_t num_episodes, const float* init_state, void* out, float* final_state,
                               void* saved, void* stream) {
    const ofrl_status s = check_sequence(ctx, in, episode_ends, num_episodes);
    if (s != OFRL_OK) return s;
    if (num_episodes == 0) return OFRL_OK;
    if (in->tokens > 0 && out == nullptr) return OFRL_EINVAL;
    if (!aligned16(out) || !aligned16(init_state) || !aligned16(final_state) ||
        (reinterpret_cast<uintptr_t>(saved) & 255u) ||
        !same_or_apart(init_state, final_state, states_bytes(ctx->shape, num_episodes)))
        return OFRL_EINVAL;
    SeqLaunch a = base_launch(ctx, in, episode_ends, num_episodes);
    a.init = init_state;
    a.out = out;
    a.final_state = final_state;
    a.saved = static_cast<uint8_t*>(saved);
    return cuda_status(launch_forward(a, static_cast<cudaStream_t>(stream)));
}

ofrl_status ofrl_delta_backward(ofrl_delta* ctx, const ofrl_delta_tokens* in, const int32_t* episode_ends,
                                int32_t num_episodes, const void* saved, const void* dout, const float* d_final,
                                const ofrl_delta_grads* grads, float* d_init, void* stream) {
    const ofrl_status s = check_sequence(ctx, in, episode_ends, num_episodes);
    if (s != OFRL_OK) return s;
    if (!ctx->backward) return OFRL_EINVAL;
    if (num_episodes == 0) return OFRL_OK;
    if (saved == nullptr || (reinterpret_cast<uintptr_t>(saved) & 255u) || grads == nullptr) return OFRL_EINVAL;
    if (!aligned16(dout) || !aligned16(d_final) || !aligned16(d_init) ||
        !same_or_apart(d_final, d_init, states_bytes(ctx->shape, num_episodes)))
        return OFRL_EINVAL;
    if (in->tokens > 0) {
        const ofrl_delta_shape& h = ctx->shape;
        const int64_t e = elem_size(h), qk = (int64_t)h.k_heads * h.k_dim, vv = (int64_t)h.v_heads * h.v_dim;
        if (!dout || !grads->dq || !grads->dk || !grads->dv || !grads->dg || !grads->dbeta) return OFRL_EINVAL;
        if (!aligned16(grads->dq) || !aligned16(grads->dk) || !aligned16(grads->dv)) return OFRL_EINVAL;
        if ((reinterpret_cast<uintptr_t>(grads->dg) | reinterpret_cast<uintptr_t>(grads->dbeta)) & (uintptr_t)(e - 1))
            return OFRL_EINVAL;
        if (!stride_ok(grads->q_stride, qk, e, true) || !stride_ok(grads->k_stride, qk, e, true) ||
            !stride_ok(grads->v_stride, vv, e, true) || !stride_ok(grads->g_stride, h.v_heads, e, false) ||
            !stride_ok(grads->beta_stride, h.v_heads, e, false))
            return OFRL_EINVAL;
    }
    SeqLaunch a = base_launch(ctx, in, episode_ends, num_episodes);
    a.saved = static_cast<uint8_t*>(const_cast<void*>(saved));
    a.dout = dout;
    a.d_final = d_final;
    a.grads = *grads;
    a.d_init = d_init;
    return cuda_status(launch_backward(a, static_cast<cudaStream_t>(stream)));
}

ofrl_status ofrl_delta_step(ofrl_delta* ctx, const ofrl_delta_tokens* in, const int32_t* slot_idx, int32_t slots,
                            const float* state_in, float* state_out, void* out, void* stream) {
    ofrl_status s = check_ctx(ctx);
    if (s == OFRL_OK) s = check_tokens(ctx, in);
    if (s != OFRL_OK) return s;
    if (slots < 0 || (slot_idx == nullptr && slots < in->tokens)) return OFRL_EINVAL;
    if (in->tokens == 0) return OFRL_OK;
    if (!out || !aligned16(out) || !aligned16(state_in) || !aligned16(state_out)) return OFRL_EINVAL;
    if (slots > 0 && (!state_in || !state_out)) return OFRL_EINVAL;
    if (!same_or_apart(state_in, state_out, states_bytes(ctx->shape, slots))) return OFRL_EINVAL;
    StepLaunch a;
    std::memset(&a, 0, sizeof(a));
    a.shape = ctx->shape;
    a.in = *in;
    a.slot_idx = slot_idx;
    a.slots = slots;
    a.state_in = state_in;
    a.state_out = state_out;
    a.out = out;
    a.status = ctx->status;
    a.num_sms = ctx->num_sms;
    return cuda_status(launch_step(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
