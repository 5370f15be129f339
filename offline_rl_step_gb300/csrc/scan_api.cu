// C entry points of the selective scan: argument checks, the context, how a
// call is cut.  Nothing here allocates except ofrl_scan_create.

#include <cstring>
#include <new>

#include "rows.cuh"
#include "scan.cuh"
#include "../../include/ofrl_selftest.h"

namespace ofrl {
namespace scan {
namespace {

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
int64_t div_up(int64_t x, int64_t m) { return (x + m - 1) / m; }

// CTAs over all channels for one form.
int blocks_of(const ofrl_scan_shape& s, int ls, int cpt) {
    return s.groups * (int)div_up(s.channels / s.groups, block_of(ls, cpt));
}
// Segments wanted for `blocks` CTAs each: `per_sm` CTAs on every SM.
int64_t wanted(int blocks, int num_sms, int per_sm) { return div_up((int64_t)num_sms * per_sm, blocks); }
// What its registers and shared memory let an SM hold.
int per_sm_of(bool backward, int cpt) { return !backward ? 4 : cpt == 4 ? 2 : 3; }

}  // namespace

// The cut of a call.  All in us, tokens in bf16 with a gate unless said otherwise.
//
// 1. Whole episodes to a segment, since those have no tails, where their number
//    divides the tokens (the host does not know their lengths) and there is a CTA for
//    every SM: 64 episodes of 256, 512 channels of 16 states read 64 (even shares 88),
//    256 of 64 118 (156), 1024 of 8 76 (105); 100 of 160, 256 of 16, trained 167 (186).
//    But a whole episode is longer than an even share, and fewer CTAs hide less
//    latency: 32 of 512, 256 of 64, read 221 (156); gradients of 1024 channels of 8
//    states for them 379 (275); so there are limits on how much longer.
// 2. Even shares in the wide form (a token's deltas and inputs are read by fewer
//    threads, its B and C serve more channels), where that makes two CTAs an SM
//    (gradients: one and a half), whatever an SM holds of that form: 16384 tokens of
//    512 channels of 16 states read 88 (narrow 111 to 116), trained 331 (358).
// 3. Even shares in the narrow one: 8 episodes of 128 to 384, 128 channels of 16
//    states, read 17 (wide 25), trained 58 (79).
// Only the narrow form where the wide one leaves a quarter more threads without a
// channel: 228 episodes of 64 to 512, 144 channels of 16 states, read 124 (wide 154),
// trained 486 (604); two groups of 72, read 143 (155).
Cut cut_of(const ofrl_scan_shape& s, int64_t tokens, int64_t episodes, int num_sms, bool backward) {
    Cut c;
    c.ls = lanes_of(s.state_dim);
    // of episodes that may all be that long, in whole tiles
    const int64_t mean = episodes > 0 && tokens % episodes == 0 && tokens / episodes % kTile == 0 ? tokens / episodes : 0;
    const int narrow = narrow_of(c.ls, backward);
    // channels that the CTAs have threads for
    auto padded = [&](int cpt) { return blocks_of(s, c.ls, cpt) * block_of(c.ls, cpt); };
    const int wide = 5 * (int64_t)padded(narrow) <= 4 * (int64_t)padded(wide_of(c.ls)) ? narrow : wide_of(c.ls);
    // an even share of the tokens for each CTA that the GPU holds
    auto share = [&](int cpt) {
        c.cpt = cpt;
        c.blocks = blocks_of(s, c.ls, cpt);
        const int64_t seg = round_up(div_up(tokens, wanted(c.blocks, num_sms, per_sm_of(backward, cpt))), kTile);
        c.seg = (int)(seg < kMinSegment ? kMinSegment : seg > kMaxSegment ? kMaxSegment : seg);
    };
    auto cut = [&](int64_t seg) {
        c.seg = (int)seg;
        const int64_t n = div_up(tokens, seg);
        c.n_seg = (int)(n > 1 ? n : 1);
    };
    // cut to whole episodes, of at most that many quarters of an even share, if there is a CTA for every SM
    auto whole = [&](int quarters) {
        if (mean <= c.seg || 4 * mean > (int64_t)quarters * c.seg || mean > kMaxSegment ||
            (int64_t)c.blocks * div_up(tokens, mean) < num_sms)
            return false;
        cut(mean);
        return true;
    };
    const int most = backward ? 5 : c.ls == 16 ? 6 : 10;
    share(wide);
    if (whole(most)) return c;
    // before even shares of the wide form: 64 of 256, 256 channels of 16 states, read 48 (63)
    share(narrow);
    if (whole(backward ? 5 : 6)) return c;
    share(wide);
    cut(c.seg);
    if (wide != narrow && 2 * (int64_t)c.blocks * c.n_seg < (backward ? 3 : 4) * num_sms) {
        share(narrow);
        if (!whole(most)) cut(c.seg);      // 64 of 256, 128 channels of 16 states, read 36 (39), trained 114 (117)
    }
    return c;
}

Work work_of(const ofrl_scan_shape& s, int64_t tokens, const Cut& c, bool backward) {
    Work w;
    int64_t o = 0;
    auto take = [&](int64_t bytes) { const int64_t at = o; o = round_up(o + bytes, 256); return at; };
    const int64_t segs = c.n_seg, states = (int64_t)s.channels * s.state_dim;
    w.tail = take(segs * states * 4);
    w.sum = take(segs * s.channels * 4);
    w.kind = take(segs * 4);
    w.dbc = w.da = w.dd = o;
    if (backward) {
        const int64_t parts = c.blocks / s.groups;
        w.dbc = take(parts > 1 ? parts * tokens * s.groups * 8 * c.ls * 4 : 0);
        w.da = take(segs * states * 4);
        w.dd = take(2 * segs * s.channels * 4);
    }
    w.total = o;
    return w;
}

// Enough for every call of at most max_tokens: for each form, at most this many
// segments, and parts for all tokens.
int64_t work_bytes(const ofrl_scan_shape& s, int64_t max_tokens, int num_sms, bool backward) {
    int64_t most = 0;
    Cut c;
    c.ls = lanes_of(s.state_dim);
    for (int back = 0; back <= (backward ? 1 : 0); ++back)
        for (int cpt = wide_of(c.ls);; cpt = narrow_of(c.ls, back != 0)) {
            c.cpt = cpt;
            c.blocks = blocks_of(s, c.ls, cpt);
            // a segment is no shorter than an even share and than kMinSegment, or it is kMaxSegment
            const int64_t even = wanted(c.blocks, num_sms, per_sm_of(back != 0, cpt)), least = div_up(max_tokens, kMinSegment),
                          longest = div_up(max_tokens, kMaxSegment);
            const int64_t few = even < least ? even : least;
            const int64_t n = longest > few ? longest : few;
            c.n_seg = (int)(n > 1 ? n : 1);
            const int64_t bytes = work_of(s, max_tokens, c, back != 0).total;
            most = bytes > most ? bytes : most;
            if (cpt == narrow_of(c.ls, back != 0)) break;
        }
    return most;
}

int64_t saved_bytes(const ofrl_scan_shape& s, int64_t tokens) {
    return div_up(tokens, kSave) * s.channels * s.state_dim * 4;
}

}  // namespace scan
}  // namespace ofrl

using namespace ofrl;
using namespace ofrl::scan;

namespace {

ofrl_status check_shape(const ofrl_scan_shape* s) {
    if (s == nullptr || s->channels < 1 || s->state_dim < 1 || s->groups < 1 || s->channels % s->groups != 0 ||
        !dtype_ok(s->dtype) || (s->softplus != 0 && s->softplus != 1))
        return OFRL_EINVAL;
    if (s->channels > 65536 || (s->channels / s->groups) % 8 != 0 || s->state_dim > 64 || s->state_dim % 4 != 0)
        return OFRL_EUNSUPPORTED;
    return OFRL_OK;
}

ofrl_status check_tokens(const ofrl_scan* ctx, const ofrl_scan_tokens* t) {
    if (t == nullptr || t->tokens < 0 || t->tokens > kMaxTokens) return OFRL_EINVAL;
    const ofrl_scan_shape& s = ctx->shape;
    if (t->a == nullptr || !aligned_to(t->a, 16) || !aligned_to(t->d, 4) || !aligned_to(t->dt_bias, 4)) return OFRL_EINVAL;
    if (t->tokens == 0) return OFRL_OK;
    const int64_t e = dtype_size(s.dtype), d = s.channels, bc = (int64_t)s.groups * s.state_dim;
    if (!rows_ok(t->x, t->x_stride, d, e) || !rows_ok(t->dt, t->dt_stride, d, e)) return OFRL_EINVAL;
    if (t->z != nullptr && !rows_ok(t->z, t->z_stride, d, e)) return OFRL_EINVAL;
    if (t->b == nullptr || t->c == nullptr || !aligned_to(t->b, e) || !aligned_to(t->c, e) ||
        !stride_ok(t->b_stride, bc) || !stride_ok(t->c_stride, bc))
        return OFRL_EINVAL;
    return OFRL_OK;
}

ofrl_status check_sequence(const ofrl_scan* ctx, const ofrl_scan_tokens* in, const int32_t* ends, int32_t episodes) {
    ofrl_status s = check_device(ctx);
    if (s == OFRL_OK) s = check_tokens(ctx, in);
    if (s != OFRL_OK) return s;
    if (episodes < 0 || (episodes > 0 && (ends == nullptr || !aligned_to(ends, 4)))) return OFRL_EINVAL;
    if (in->tokens > 0 && episodes == 0) return OFRL_EINVAL;
    if (in->tokens > ctx->max_tokens || episodes > ctx->max_episodes) return OFRL_EINVAL;
    return OFRL_OK;
}

scan::Launch base_launch(const ofrl_scan* ctx, const ofrl_scan_tokens* in, const int32_t* ends, int32_t episodes,
                         const Cut& c, bool backward) {
    scan::Launch a;
    std::memset(&a, 0, sizeof(a));
    a.shape = ctx->shape;
    a.in = *in;
    a.ends = ends;
    a.episodes = episodes;
    a.status = ctx->status;
    const Work w = work_of(ctx->shape, in->tokens, c, backward);
    a.tail = reinterpret_cast<float*>(ctx->work + w.tail);
    a.sum = reinterpret_cast<float*>(ctx->work + w.sum);
    a.kind = reinterpret_cast<int32_t*>(ctx->work + w.kind);
    a.dbc = reinterpret_cast<float*>(ctx->work + w.dbc);
    a.da = reinterpret_cast<float*>(ctx->work + w.da);
    a.dd = reinterpret_cast<float*>(ctx->work + w.dd);
    a.seg = c.seg;
    a.n_seg = c.n_seg;
    a.blocks = c.blocks;
    return a;
}

}  // namespace

extern "C" {

int64_t ofrl_scan_workspace_bytes(const ofrl_scan_shape* shape, int64_t max_tokens, int32_t max_episodes,
                                  int32_t backward) {
    if (check_shape(shape) != OFRL_OK || !counts_ok(max_tokens, max_episodes) || (backward != 0 && backward != 1))
        return -1;
    int device = 0;
    const int sms = current_sms(&device);
    return 256 + work_bytes(*shape, max_tokens, sms > 0 ? sms : 1, backward != 0);
}

int64_t ofrl_scan_saved_bytes(const ofrl_scan_shape* shape, int64_t tokens) {
    if (check_shape(shape) != OFRL_OK || !counts_ok(tokens, 0)) return -1;
    return saved_bytes(*shape, tokens);
}

ofrl_status ofrl_scan_create(const ofrl_scan_shape* shape, int64_t max_tokens, int32_t max_episodes, int32_t backward,
                             ofrl_scan** out) {
    if (out == nullptr) return OFRL_EINVAL;
    *out = nullptr;
    const ofrl_status s = check_shape(shape);
    if (s != OFRL_OK) return s;
    if (!counts_ok(max_tokens, max_episodes) || (backward != 0 && backward != 1)) return OFRL_EINVAL;
    ofrl_scan* ctx = new (std::nothrow) ofrl_scan;
    if (ctx == nullptr) return OFRL_ECUDA;
    std::memset(ctx, 0, sizeof(*ctx));
    ctx->num_sms = current_sms(&ctx->device);
    ctx->shape = *shape;
    ctx->max_tokens = max_tokens;
    ctx->max_episodes = max_episodes;
    ctx->backward = backward;
    if (ctx->num_sms > 0) ctx->bytes = 256 + work_bytes(*shape, max_tokens, ctx->num_sms, backward != 0);
    if (ctx->num_sms == 0 || take_memory(&ctx->base, ctx->bytes) != cudaSuccess) {
        delete ctx;
        return OFRL_ECUDA;
    }
    ctx->status = static_cast<int32_t*>(ctx->base);
    ctx->work = static_cast<uint8_t*>(ctx->base) + 256;
    *out = ctx;
    return OFRL_OK;
}

ofrl_status ofrl_scan_destroy(ofrl_scan* ctx) { return release_memory(ctx); }

ofrl_status ofrl_scan_poll_status(ofrl_scan* ctx, void* stream, int32_t* words_out) {
    return poll_words(ctx, stream, words_out);
}

ofrl_status ofrl_scan_forward(ofrl_scan* ctx, const ofrl_scan_tokens* in, const int32_t* episode_ends,
                              int32_t num_episodes, const float* init_state, void* out, int64_t out_stride,
                              float* final_state, void* saved, void* stream) {
    const ofrl_status s = check_sequence(ctx, in, episode_ends, num_episodes);
    if (s != OFRL_OK) return s;
    if (num_episodes == 0) return OFRL_OK;
    if (in->tokens > 0 && !rows_ok(out, out_stride, ctx->shape.channels, dtype_size(ctx->shape.dtype))) return OFRL_EINVAL;
    if (!aligned_to(init_state, 16) || !aligned_to(final_state, 16) || !aligned_to(saved, 16)) return OFRL_EINVAL;
    const int64_t state = (int64_t)num_episodes * ctx->shape.channels * ctx->shape.state_dim * 4;
    if (overlap(init_state, state, final_state, state)) return OFRL_EINVAL;
    const Cut c = cut_of(ctx->shape, in->tokens, num_episodes, ctx->num_sms, false);
    scan::Launch a = base_launch(ctx, in, episode_ends, num_episodes, c, false);
    a.init = init_state;
    a.out = out;
    a.out_stride = out_stride;
    a.final_state = final_state;
    a.saved = static_cast<float*>(saved);
    return cuda_status(launch_forward(a, c, static_cast<cudaStream_t>(stream)));
}

ofrl_status ofrl_scan_backward(ofrl_scan* ctx, const ofrl_scan_tokens* in, const int32_t* episode_ends,
                               int32_t num_episodes, const float* init_state, const void* saved, const void* dout,
                               int64_t dout_stride, const float* d_final, const ofrl_scan_grads* grads, float* d_init,
                               void* stream) {
    const ofrl_status s = check_sequence(ctx, in, episode_ends, num_episodes);
    if (s != OFRL_OK) return s;
    if (!ctx->backward || grads == nullptr) return OFRL_EINVAL;
    if (grads->da == nullptr || !aligned_to(grads->da, 16) || !aligned_to(grads->dd, 4) || !aligned_to(grads->ddt_bias, 4))
        return OFRL_EINVAL;
    if (!aligned_to(init_state, 16) || !aligned_to(saved, 16) || !aligned_to(d_final, 16) || !aligned_to(d_init, 16))
        return OFRL_EINVAL;
    const ofrl_scan_shape& h = ctx->shape;
    const int64_t state = (int64_t)num_episodes * h.channels * h.state_dim * 4;
    if (overlap(init_state, state, d_init, state) || overlap(d_final, state, d_init, state)) return OFRL_EINVAL;
    if (in->tokens > 0) {
        const int64_t e = dtype_size(h.dtype), d = h.channels, bc = (int64_t)h.groups * h.state_dim;
        if (saved == nullptr || !rows_ok(dout, dout_stride, d, e)) return OFRL_EINVAL;
        if (!rows_ok(grads->dx, grads->x_stride, d, e) || !rows_ok(grads->ddt, grads->dt_stride, d, e)) return OFRL_EINVAL;
        if ((grads->dz == nullptr) != (in->z == nullptr) ||
            (in->z != nullptr && !rows_ok(grads->dz, grads->z_stride, d, e)))
            return OFRL_EINVAL;
        if (grads->db == nullptr || grads->dc == nullptr || !aligned_to(grads->db, e) || !aligned_to(grads->dc, e) ||
            !stride_ok(grads->b_stride, bc) || !stride_ok(grads->c_stride, bc))
            return OFRL_EINVAL;
    }
    const Cut c = cut_of(h, in->tokens, num_episodes, ctx->num_sms, true);
    scan::Launch a = base_launch(ctx, in, episode_ends, num_episodes, c, true);
    a.init = init_state;
    a.saved = static_cast<float*>(const_cast<void*>(saved));
    a.dout = dout;
    a.dout_stride = dout_stride;
    a.d_final = d_final;
    a.grads = *grads;
    a.d_init = d_init;
    return cuda_status(launch_backward(a, c, static_cast<cudaStream_t>(stream)));
}

ofrl_status ofrl_scan_step(ofrl_scan* ctx, const ofrl_scan_tokens* in, const int32_t* slot_idx, int32_t slots,
                           const float* state_in, float* state_out, void* out, int64_t out_stride, void* stream) {
    ofrl_status s = check_device(ctx);
    if (s == OFRL_OK) s = check_tokens(ctx, in);
    if (s != OFRL_OK) return s;
    if (slots < 0 || !aligned_to(slot_idx, 4) || (slot_idx == nullptr && slots < in->tokens)) return OFRL_EINVAL;
    if (in->tokens == 0) return OFRL_OK;
    if (!rows_ok(out, out_stride, ctx->shape.channels, dtype_size(ctx->shape.dtype))) return OFRL_EINVAL;
    if (!aligned_to(state_in, 16) || !aligned_to(state_out, 16)) return OFRL_EINVAL;
    if (slots > 0 && (!state_in || !state_out)) return OFRL_EINVAL;
    if (!same_or_apart(state_in, state_out, (int64_t)slots * ctx->shape.channels * ctx->shape.state_dim * 4))
        return OFRL_EINVAL;
    scan::StepLaunch a;
    std::memset(&a, 0, sizeof(a));
    a.shape = ctx->shape;
    a.in = *in;
    a.slot_idx = slot_idx;
    a.slots = slots;
    a.state_in = state_in;
    a.state_out = state_out;
    a.out = out;
    a.out_stride = out_stride;
    a.status = ctx->status;
    a.num_sms = ctx->num_sms;
    const int64_t four = 4 * dtype_size(ctx->shape.dtype);
    a.whole_states = aligned_to(in->b, four) && aligned_to(in->c, four) && in->b_stride % 4 == 0 && in->c_stride % 4 == 0;
    return cuda_status(launch_step(a, static_cast<cudaStream_t>(stream)));
}

ofrl_status ofrl_selftest_scan_cut(const ofrl_scan_shape* shape, int64_t tokens, int32_t episodes, int64_t max_tokens,
                                   int32_t num_sms, int32_t backward, int64_t* out) {
    const ofrl_status s = check_shape(shape);
    if (s != OFRL_OK) return s;
    if (!counts_ok(tokens, episodes) || !counts_ok(max_tokens, 0) || num_sms < 1 || (backward != 0 && backward != 1) ||
        out == nullptr)
        return OFRL_EINVAL;
    const Cut c = cut_of(*shape, tokens, episodes, num_sms, backward != 0);
    out[0] = c.ls;
    out[1] = c.cpt;
    out[2] = c.blocks;
    out[3] = c.seg;
    out[4] = c.n_seg;
    out[5] = work_of(*shape, tokens, c, backward != 0).total;
    out[6] = work_bytes(*shape, max_tokens, num_sms, backward != 0);
    return OFRL_OK;
}

}  // extern "C"
