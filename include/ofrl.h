/*
 * ofrl.h -- C ABI of the GB300 (sm_103a) fused offline-RL train step:
 * HER batch relabel followed by an IQL value-network update with budgeted
 * per-source gradient clipping and Adam.
 *
 * Conventions shared by every entry point
 * ----------------------------------------
 *  - Pointers named in a comment as "device" are CUDA device pointers
 *    (or managed memory) on the current device; the caller owns every buffer.
 *    ofrl_train_step's q, loss_out and norms_out may also point into
 *    page-locked host memory (cudaHostAlloc / cudaHostRegister): the
 *    relabel launch then copies Q over the host link (NVLink-C2C on
 *    Grace-Blackwell) into the workspace while the previous step's
 *    optimizer kernel still runs, and the optimizer writes the loss and
 *    norms in place, instead of copies on the stream.
 *    The context owns only its workspace (gradient partials, reduction
 *    scratch, the status word), sized once at ofrl_create.  No call after
 *    ofrl_create allocates.
 *  - Every compute call is asynchronous on `stream` (a cudaStream_t; NULL =
 *    the legacy default stream) and never synchronises the host, except
 *    ofrl_poll_status.
 *  - Shape, pointer-alignment and unsupported-configuration errors are
 *    detected on the host before anything is launched and return
 *    OFRL_EINVAL / OFRL_EUNSUPPORTED with nothing written.  A failed launch
 *    returns OFRL_ECUDA.  Anomalies only visible on the device (non-finite
 *    gradient elements skipped by Adam, out-of-range actions or indices) are
 *    counted in the context's status word, read by ofrl_poll_status.
 *  - Floating-point buffers are fp32, row-major.  Index buffers are int32.
 *  - Results are deterministic: no floating-point atomics; every reduction
 *    runs in a fixed order, so two identical calls give identical bits.
 *  - One context must not be used by two calls that overlap on the GPU
 *    (its workspace is shared by every call); use one context per stream.
 *
 * Notation: B batch, S state_dim, g goal_dim, H hidden, A num_actions,
 * P = H*S + H + H*H + H + H + 1 (V parameter count).  The flat V parameter
 * and gradient layout is W1[H,S], b1[H], W2[H,H], b2[H], W3[1,H], b3[1]
 * ("GPU IQL + HER Porting Plan", "CUDA Kernel: iql_value_kernel.cu",
 * parameter layout: w_v1, b_v1, w_v2, b_v2, w_vout, b_vout); every linear
 * layer computes y = x W^T + b.
 */
#ifndef OFRL_H
#define OFRL_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t ofrl_status;
enum {
    OFRL_OK = 0,
    OFRL_EINVAL = -1,        /* bad argument: null pointer, size, stride, alignment */
    OFRL_EUNSUPPORTED = -2,  /* valid request the library does not implement (e.g. H not in {64,128,256}) */
    OFRL_ECUDA = -3,         /* a CUDA runtime call or launch failed */
    OFRL_ETIMEOUT = -4       /* reserved: a bounded device-side wait gave up */
};

/* HER donor strategies ("GPU IQL + HER Porting Plan", "Donor Index
 * Generation"; the string map "final" / "future" / anything else -> Random
 * is in "Config Wiring" of the HER part).  EPISODE is named in "HER (CPU)"
 * item 5 without a definition: here, as in the HER paper's "episode"
 * strategy, the donor is uniform over the source's whole episode. */
enum { OFRL_HER_FINAL = 0, OFRL_HER_FUTURE = 1, OFRL_HER_RANDOM = 2, OFRL_HER_EPISODE = 3 };

/* GEMM operand precision.  FP32: fp32 operands and accumulation.  BF16:
 * GEMM operands rounded to bf16 (round-to-nearest-even), fp32 accumulation,
 * fp32 master weights, fp32 epilogues (the twin-network workload). */
enum { OFRL_PREC_FP32 = 0, OFRL_PREC_BF16 = 1 };

/* Device status word, read by ofrl_poll_status (counts since the last poll). */
enum {
    OFRL_STAT_NONFINITE_GRAD = 0,  /* gradient elements Adam skipped as non-finite */
    OFRL_STAT_BAD_ACTION = 1,      /* batch actions outside [0, A) (treated as action 0) */
    OFRL_STAT_BAD_INDEX = 2,       /* episode boundary lookups that fell outside the buffer */
    OFRL_STAT_TIMEOUT = 3,         /* bounded device waits that gave up */
    OFRL_STAT_SANITIZED = 4,       /* gradient-source elements counted as 0 (ofrl_opt.sanitize_sources) */
    OFRL_STAT_WORDS = 8
};

typedef struct ofrl_ctx ofrl_ctx;

/* Replay buffer, structure of arrays, all device, read only
 * ("GPU IQL + HER Porting Plan", "GPU PER buffer": states [capacity,
 * state_dim], next_states, actions, rewards, dones; "Episode Boundary
 * Tracking on GPU": an episode boundary array). */
typedef struct {
    const float* states;         /* [capacity, state_stride] */
    const float* next_states;    /* [capacity, state_stride] */
    const int32_t* actions;      /* [capacity] */
    const float* rewards;        /* [capacity] */
    const float* dones;          /* [capacity] */
    const int32_t* episode_ends; /* [num_episodes] exclusive ends, strictly ascending,
                                    last == capacity; needed by FINAL and FUTURE only */
    int64_t capacity;            /* 1 .. 2^31-1 transitions */
    int32_t num_episodes;
    int32_t state_dim;           /* S */
    int32_t state_stride;        /* row stride in floats, >= S, multiple of 4 (16-byte rows) */
    int32_t goal_dim;            /* g: the goal is the first g state elements, 1 <= g <= S */
} ofrl_replay;

/* HER batch assembly ("How HER Interacts with GPU PER"): rows
 * [0, batch - her_count) are normal rows, rows [batch - her_count, batch)
 * are relabelled.  her_count = floor(batch * her_ratio) is the caller's. */
typedef struct {
    int32_t batch;           /* B >= 1 */
    int32_t her_count;       /* 0 .. B */
    int32_t strategy;        /* OFRL_HER_* */
    float goal_threshold;    /* reward +1 if goal distance < threshold, else -0.01 (pages: 0.01) */
    uint64_t seed;           /* counter-based RNG key (SplitMix64, see ofrl_her_relabel) */
} ofrl_her_cfg;

/* Relabelled batch, all device, written by ofrl_her_relabel / ofrl_train_step. */
typedef struct {
    float* states;        /* [B, stride] */
    float* next_states;   /* [B, stride] */
    int32_t* actions;     /* [B] */
    float* rewards;       /* [B] */
    float* dones;         /* [B] */
    int32_t* src_idx;     /* [B] source transition of each row */
    int32_t* donor_idx;   /* [B] goal donor of each row, -1 for normal rows */
    int32_t stride;       /* row stride in floats, >= S, multiple of 4 */
} ofrl_batch;

/* V network shape. */
typedef struct {
    int32_t state_dim;    /* S, 1 .. 64 */
    int32_t hidden;       /* H, one of 64, 128, 256 */
    int32_t num_actions;  /* A, 1 .. 16 */
    int32_t prec;         /* OFRL_PREC_* */
} ofrl_vshape;

/* One V network's trainable state, device buffers of P floats.  `t` is
 * the Adam step counter (host side); ofrl_train_step increments it before
 * the Adam phase, so the first step runs with t = 1.  `target`: the
 * network's target copy ("GPU IQL + HER Porting Plan", "Rust Integration:
 * gpu_iql_trainer.rs", target_ema_update: EMA target update for the V
 * network, Polyak averaging; step 4 of "Where in the Training Loop IQL Gets
 * Called"), or NULL; when set, ofrl_train_step updates it in the Adam pass,
 * after the weights: target = (1 - polyak) target + polyak params. */
typedef struct {
    float* params;
    float* m;
    float* v;
    int32_t t;
    float tau;            /* expectile, 0 < tau < 1 */
    float* target;        /* device [P] or NULL */
    float polyak;         /* 0 <= polyak <= 1 (read when target != NULL) */
} ofrl_vnet;

/* Optimiser and policy hyper-parameters ("GPU IQL + HER Porting Plan",
 * IqlGpuConfig fields lr, beta1, beta2, epsilon, weight_decay,
 * max_grad_norm; beta is the advantage temperature). */
typedef struct {
    float lr, beta1, beta2, eps, weight_decay;
    float max_grad_norm;  /* > 0; +inf disables every clip */
    float beta;           /* advantage temperature */
    float budget[4];      /* budget fractions, primary first (pages: 0.70, 0.15, 0.10, 0.05) */
    float alpha[4];       /* SAXPY coefficient per source, primary first (1.0 each) */
    /* "DQN Backward-Path NaN Audit": a bound on |weight| applied in the Adam
     * kernel after each update (0 disables it) ... */
    float weight_clamp_max_abs;
    /* ... and the SAXPY's isfinite guard: 1 counts non-finite elements of
     * every gradient source as 0 (in the source norms, the Gram matrix and
     * the combination; counted in OFRL_STAT_SANITIZED); 0 leaves them. */
    int32_t sanitize_sources;
} ofrl_opt;

/* ---- context -------------------------------------------------------- */

/* Create a context for V networks of `shape`, batches up to max_batch rows
 * and up to max_nets (1 or 2) networks per step.  The only allocating call.
 * Binds to the current CUDA device.  Returns OFRL_EINVAL / OFRL_EUNSUPPORTED
 * for bad shapes, OFRL_ECUDA if allocation fails; *out is NULL on error. */
ofrl_status ofrl_create(const ofrl_vshape* shape, int32_t max_batch, int32_t max_nets,
                        ofrl_ctx** out);

/* Free the context (synchronises the device first).  NULL is a no-op. */
ofrl_status ofrl_destroy(ofrl_ctx* ctx);

/* Copy the device status word (OFRL_STAT_WORDS int32 counters) to the host
 * array `words_out` and clear it.  Synchronises `stream`. */
ofrl_status ofrl_poll_status(ofrl_ctx* ctx, void* stream, int32_t* words_out);

/* Human-readable name of a status code (static storage). */
const char* ofrl_status_string(ofrl_status s);

/* Number of bytes of device workspace ofrl_create reserves for these sizes. */
int64_t ofrl_workspace_bytes(const ofrl_vshape* shape, int32_t max_batch, int32_t max_nets);

/* ---- the hot-path operations ----------------------------------------- */

/* HER index sampling + gather + relabel ("GPU IQL + HER Porting Plan",
 * "CUDA Kernel: her_relabel_kernel.cu" and "Donor Index Generation").
 * For every row b: src = below(draw(seed, step*2^32 + 2b), capacity).  For a
 * HER row the donor is: FINAL episode_end(src) - 1; FUTURE src + 1 +
 * below(draw(seed, step*2^32 + 2b + 1), episode_end(src) - src - 1), or src
 * itself when src is its episode's last transition; RANDOM
 * below(draw(seed, ...2b + 1), capacity); EPISODE episode_start(src) +
 * below(draw(seed, ...2b + 1), episode_end(src) - episode_start(src)).
 * episode_end(i) is the first entry of episode_ends above i (binary search),
 * episode_start(i) the entry before it (0 for the first episode).  draw(k, n) is output n+1
 * of SplitMix64 seeded with k; below(r, n) = ((r >> 32) * n) >> 32.
 * Row output: states/next_states/action/reward/done of src; for HER rows the
 * first g elements of both states are replaced by next_states[donor, :g]
 * and the reward is +1.0f if the fp32 distance between next_states[src, :g]
 * and next_states[donor, :g] (summed in order without fused multiply-add,
 * IEEE sqrtf) is below goal_threshold, else -0.01f.  Columns
 * [S, stride) of the output rows are copied from the source rows.
 * Writes every field of `out`. */
ofrl_status ofrl_her_relabel(ofrl_ctx* ctx, const ofrl_replay* replay, const ofrl_her_cfg* her,
                             uint64_t step, const ofrl_batch* out, void* stream);

/* The relabel with the caller's sources ("GPU IQL + HER Porting Plan", "How
 * HER Interacts with GPU PER": normal rows and the HER rows' sources come
 * from the PER sampler; the HER rows' importance weights are 1, no PER
 * bias).  src_idx: device [batch] source of every row (normal rows first,
 * then the her_count HER rows; outside [0, capacity) is clamped and counted
 * in OFRL_STAT_BAD_INDEX).  is_weights: device [batch] or NULL (weight 1).
 * is_weights_out: device [batch] or NULL: the normal rows' weights, 1 for
 * HER rows.  Donors, rewards and the copies as ofrl_her_relabel. */
ofrl_status ofrl_her_relabel_sources(ofrl_ctx* ctx, const ofrl_replay* replay, const ofrl_her_cfg* her,
                                     uint64_t step, const int32_t* src_idx, const float* is_weights,
                                     const ofrl_batch* out, float* is_weights_out, void* stream);

/* Episode-boundary maintenance on the device ("GPU IQL + HER Porting
 * Plan", "Episode Boundary Tracking on GPU": each finished episode's end is
 * appended to a GPU-resident boundary array that grows as episodes
 * complete).  n new transitions were stored at buffer positions
 * first_index .. first_index + n - 1 with done flags dones[0 .. n) (device);
 * for every i with dones[i] != 0 the exclusive end first_index + i + 1 is
 * appended to episode_ends (device, max_episodes entries) after the
 * *num_episodes (device int32) already there, in ascending order, and
 * *num_episodes grows by their number.  Ends that do not fit are dropped and
 * counted in OFRL_STAT_BAD_INDEX.  first_index + n <= 2^31 - 1. */
ofrl_status ofrl_episode_ends_append(ofrl_ctx* ctx, const float* dones, int64_t first_index, int32_t n,
                                     int32_t* episode_ends, int32_t* num_episodes, int32_t max_episodes,
                                     void* stream);

/* V forward + expectile loss + V backward ("GPU IQL + HER Porting Plan",
 * "IQL (CPU)" items 1-2 and "CUDA Kernel: iql_value_kernel.cu").
 * states: device [batch, state_stride] (columns >= S ignored);
 * q_taken: device [batch], Q(s, a_taken); params: device [P].
 * Outputs (device): v_out [batch] = V(s); loss_out [1] =
 * mean(w (q - V)^2), w = tau if q - V >= 0 else 1 - tau; grad_out [P] =
 * dloss/dparams (overwritten, not accumulated).  batch <= max_batch. */
ofrl_status ofrl_iql_value_fwd_bwd(ofrl_ctx* ctx, const float* params, const float* states,
                                   int32_t state_stride, int32_t batch, const float* q_taken,
                                   float tau, float* v_out, float* loss_out, float* grad_out,
                                   void* stream);

/* V forward only, the network's value of each state ("GPU IQL + HER
 * Porting Plan", "Rust Integration: gpu_iql_trainer.rs", forward_values:
 * a forward-only pass of the V network, result kept on the device).
 * params: device [P] (the online or the target network); states: device
 * [batch, state_stride] (columns >= S ignored).  v_out: device [batch].
 * 1 <= batch <= max_batch; asynchronous on `stream`.  Runs on the tensor
 * cores (a weight-pack launch, then one CTA per 128-row tile: G1, h1, G2,
 * V) when ofrl_vnet_path(ctx, 1) is OFRL_VNET_TC_FUSED and the states are
 * 16-byte aligned with state_stride a multiple of 4; else on the CUDA
 * cores.  Uses the context's weight-image workspace, so calls on one
 * context must not overlap. */
ofrl_status ofrl_forward_values(ofrl_ctx* ctx, const float* params, const float* states,
                                int32_t state_stride, int32_t batch, float* v_out, void* stream);

/* IQL bootstrap target for the Q loss ("GPU IQL + HER Porting Plan", "IQL
 * modifies the target computation": r + gamma V(s') in place of the
 * max-over-actions target): target_out[b] = rewards[b] + gamma (1 - dones[b])
 * V(next_states[b]) with V from `params` (terminal rows bootstrap nothing).
 * rewards, dones: device [batch] (e.g. the relabelled batch's); v_next_out:
 * device [batch] or NULL, receives V(s').  gamma in [0, 1].  Same
 * implementation choice as ofrl_forward_values. */
ofrl_status ofrl_iql_target(ofrl_ctx* ctx, const float* params, const float* next_states,
                            int32_t state_stride, const float* rewards, const float* dones,
                            int32_t batch, float gamma, float* v_next_out, float* target_out,
                            void* stream);

/* Expectile loss alone ("IQL (CPU)" item 2): q_taken, v device [batch];
 * loss_out device [1] = mean(w d^2), d = q - v; dv_out device [batch] or
 * NULL: dloss/dv = -2 w d / batch.  batch >= 1. */
ofrl_status ofrl_expectile_loss(ofrl_ctx* ctx, const float* q_taken, const float* v,
                                int32_t batch, float tau, float* loss_out, float* dv_out,
                                void* stream);

/* Advantage-weighted policy ("IQL (CPU)" item 3): q device [batch,
 * num_actions], v device [batch]; pi_out device [batch, num_actions] =
 * softmax(beta * clamp(q - v, -10, 10)) with max-subtraction; argmax_out
 * device [batch] or NULL: lowest index of the row's largest pi. */
ofrl_status ofrl_adv_weighted_policy(ofrl_ctx* ctx, const float* q, const float* v,
                                     int32_t batch, int32_t num_actions, float beta,
                                     float* pi_out, int32_t* argmax_out, void* stream);

/* Budgeted clipped SAXPY ("Gradient Stability -- Multi-Task Gradient
 * Isolation + Full Spectral Norm", "Proper design" and Task 1 Step 5):
 * grad_out = sum_k alpha[k] * s_k * src[k], s_k = (n_k > c_k && n_k > 0) ?
 * c_k / n_k : 1, n_k = ||src[k]||, c_k = budget_frac[k] * max_grad_norm.
 * src: host array of n_src (1..4) device pointers to [n] floats (src[0] is
 * the primary); budget_frac, alpha: host arrays of n_src.  grad_out: device
 * [n] (may alias no source).  norms_out: device [n_src + 1] =
 * n_0 .. n_{n_src-1}, ||grad_out||. */
ofrl_status ofrl_budgeted_clip_saxpy(ofrl_ctx* ctx, const float* const* src,
                                     const float* budget_frac, const float* alpha,
                                     int32_t n_src, int64_t n, float max_grad_norm,
                                     float* grad_out, float* norms_out, void* stream);

/* Adam with the safety clip ("DQN Backward-Path NaN Audit", Adam kernel
 * findings; "GPU IQL + HER Porting Plan", "CUDA Kernel: iql_adam_kernel.cu"):
 * s = (n > mgn && n > 0) ? mgn / n : 1 with n = *grad_norm (device scalar,
 * or NULL to compute ||g|| here); per element g' = s * g[i]; a non-finite
 * g' leaves p, m, v unchanged and is counted in the status word; else
 * m = b1 m + (1-b1) g', v = b2 v + (1-b2) g'^2, p -= lr (m/(1-b1^t) /
 * (sqrt(v/(1-b2^t)) + eps) + weight_decay p), then p clamped to
 * [-w, w] with w = opt->weight_clamp_max_abs when w > 0.  t >= 1. */
ofrl_status ofrl_adam_step(ofrl_ctx* ctx, float* p, const float* g, float* m, float* v,
                           int64_t n, int32_t t, const ofrl_opt* opt, const float* grad_norm,
                           void* stream);

/* Polyak (EMA) update of a target network ("GPU IQL + HER Porting Plan",
 * "Rust Integration: gpu_iql_trainer.rs", target_ema_update):
 * target[i] = (1 - polyak) target[i] + polyak params[i], i < n.  Device
 * buffers; 0 <= polyak <= 1.  Needs no context. */
ofrl_status ofrl_target_ema(const float* params, float* target, int64_t n, float polyak, void* stream);

/* The fused train step: relabel -> per network {V fwd, expectile loss on
 * Q[b, action_b], policy, V bwd -> primary gradient g0; budgeted combine of
 * g0 (budget[0]) and the network's aux sources (budget[1..]); t += 1; Adam}.
 * q: device [B, A]; nets: host array of n_nets (1 or 2) networks sharing
 * the batch and Q; aux_src: host array of n_nets * n_aux device pointers
 * (network-major) to [P] floats, or NULL when n_aux == 0 (0..3).
 * Outputs (device, each may be NULL except batch): v_out [n_nets, B],
 * pi_out [n_nets, B, A], argmax_out [n_nets, B], loss_out [n_nets],
 * norms_out [n_nets, 5] (n_0..n_3 pre-clip source norms, 0 for absent
 * sources, then the combined norm), grad_out [n_nets, P] (the primary
 * gradient g0).  Increments nets[k].t on the host.
 * When the previous launch of this context on `stream` was a train step, the
 * relabel of this step's batch starts while that step's optimizer kernel
 * still runs (it reads only the replay buffer and, when q is in host memory,
 * q, and writes only the batch and the context's copy of q; the V kernel
 * still waits for both).  Writes to the replay buffer or q in between by
 * ordinary kernels or copies are ordered as usual; a kernel of the caller's
 * that lets its dependents launch early (programmatic dependent launch)
 * must not write them right before a step. */
ofrl_status ofrl_train_step(ofrl_ctx* ctx, const ofrl_replay* replay, const ofrl_her_cfg* her,
                            uint64_t step, const ofrl_batch* batch, const float* q,
                            ofrl_vnet* nets, int32_t n_nets, const ofrl_opt* opt,
                            const float* const* aux_src, int32_t n_aux,
                            float* v_out, float* pi_out, int32_t* argmax_out, float* loss_out,
                            float* norms_out, float* grad_out, void* stream);

/* Kernel launches one ofrl_train_step on this context makes for `rows`
 * batch rows and n_nets networks writing into `batch` (no counterpart on the
 * pages: a planning aid for launch accounting and graph capture): relabel,
 * one V kernel (two on the layered tensor-core path), then reduce and Adam
 * as one cooperative launch when its grid fits on the device at once, else
 * two.  Returns 0 for invalid arguments.  Host only; launches nothing. */
int32_t ofrl_train_step_kernels(const ofrl_ctx* ctx, const ofrl_batch* batch, int32_t rows, int32_t n_nets);

/* ---- V forward/backward implementations --------------------------------
 * The batch x hidden GEMMs of the value network ("GPU IQL + HER Porting
 * Plan", "CUDA Kernel: iql_value_kernel.cu"; five GEMMs per network and
 * step) run in one of three ways, all with the same results to fp32
 * rounding (no counterpart on the pages, which use cuBLAS):
 *   TC_FUSED   H = 128, S <= 64: one CTA per 128-row tile runs all five
 *              GEMMs on the tensor cores (tcgen05, accumulators in TMEM);
 *   TC_LAYERED H = 128 or 256, S < 64: per tile the forward and the
 *              backward to dz1 on the tensor cores with operands streamed by
 *              TMA, then the weight gradients split over K-ranges of the
 *              batch (two kernels);
 *   CUDA_CORES every H in {64, 128, 256}.
 * AUTO (the default) takes TC_FUSED for H = 128, TC_LAYERED for H = 256 and
 * CUDA_CORES otherwise, falling back to CUDA_CORES where a choice does not
 * apply to a call (e.g. unaligned states in a standalone call).
 * ofrl_select_vnet_path sets the context's choice: OFRL_EUNSUPPORTED when
 * the shape (or the driver, for the layered path's tensor maps) does not
 * allow it, OFRL_EINVAL for an unknown value.  ofrl_vnet_path returns the
 * implementation a train step of n_nets networks takes (an OFRL_VNET_*
 * value, never AUTO), or -1 for invalid arguments.  Host only. */
enum { OFRL_VNET_AUTO = 0, OFRL_VNET_TC_FUSED = 1, OFRL_VNET_TC_LAYERED = 2, OFRL_VNET_CUDA_CORES = 3 };
ofrl_status ofrl_select_vnet_path(ofrl_ctx* ctx, int32_t path);
int32_t ofrl_vnet_path(const ofrl_ctx* ctx, int32_t n_nets);

/* ---- the step as a CUDA graph ------------------------------------------
 * "Phase 2: Multi-Stream Graph Parallelism" runs the trainers' step as a
 * captured CUDA graph.  ofrl_step_graph_create captures one ofrl_train_step
 * with these arguments (all of them checked as ofrl_train_step checks them;
 * nothing runs) and instantiates it.  ofrl_step_graph_launch replays it on
 * `stream` as the step `step`: the relabel uses `step`; q ([B, A], device
 * or, as for ofrl_train_step, page-locked host memory; NULL keeps the
 * previous one) and aux_src (host array of n_nets * n_aux
 * device pointers, or NULL to keep the previous ones) replace the captured
 * pointers; each network's t advances by one in the caller's `nets` array
 * (which must outlive the graph), exactly as ofrl_train_step would.  Every
 * other buffer is the one given at creation.  One graph launch on the host
 * per step.  The graph uses the context's workspace: do not interleave its
 * replays with other calls on the context from another stream.  Profiling
 * hooks (ofrl_profile_begin) must be off while creating one. */
typedef struct ofrl_step_graph ofrl_step_graph;
ofrl_status ofrl_step_graph_create(ofrl_ctx* ctx, const ofrl_replay* replay, const ofrl_her_cfg* her,
                                   const ofrl_batch* batch, const float* q, ofrl_vnet* nets, int32_t n_nets,
                                   const ofrl_opt* opt, const float* const* aux_src, int32_t n_aux,
                                   float* v_out, float* pi_out, int32_t* argmax_out, float* loss_out,
                                   float* norms_out, float* grad_out, ofrl_step_graph** out);
ofrl_status ofrl_step_graph_launch(ofrl_step_graph* graph, uint64_t step, const float* q,
                                   const float* const* aux_src, void* stream);
ofrl_status ofrl_step_graph_destroy(ofrl_step_graph* graph);

/* The step graph with its host I/O inside (no counterpart on the pages): as
 * ofrl_step_graph_create, plus a copy of q_host (pinned host [B, A]) into
 * the device q before the kernels and copies of loss_out and norms_out into
 * loss_host ([n_nets]) and norms_host ([n_nets, 5]) after them, as nodes of
 * the graph; any of the three may be NULL (no copy).  Host buffers must be
 * page-locked (cudaHostAlloc / cudaHostRegister).  ofrl_step_graph_launch_io
 * replays it as step `step` with this step's host buffers (NULL keeps the
 * previous one): one graph launch does the copy-in, the step and the
 * copy-out.  The results are in the host buffers once `stream` has reached
 * the launch (synchronise or wait on an event).  ofrl_step_graph_destroy
 * releases it. */
ofrl_status ofrl_step_graph_create_io(ofrl_ctx* ctx, const ofrl_replay* replay, const ofrl_her_cfg* her,
                                      const ofrl_batch* batch, float* q, ofrl_vnet* nets, int32_t n_nets,
                                      const ofrl_opt* opt, const float* const* aux_src, int32_t n_aux,
                                      float* v_out, float* pi_out, int32_t* argmax_out, float* loss_out,
                                      float* norms_out, float* grad_out, const float* q_host, float* loss_host,
                                      float* norms_host, ofrl_step_graph** out);
ofrl_status ofrl_step_graph_launch_io(ofrl_step_graph* graph, uint64_t step, const float* q_host,
                                      const float* const* aux_src, float* loss_host, float* norms_host,
                                      void* stream);

/* ---- allocation-free variant (no counterpart in the method's pages) ---- */

/* Some callers may not allocate device memory: code whose GPU memory is
 * handed out by a host application's or framework's own pool (direct
 * cudaMalloc forbidden), code recorded into a CUDA graph under the global
 * capture mode (cudaMalloc is refused there), and latency-critical loops that
 * cannot take cudaMalloc's implicit device synchronisation.  ofrl_create
 * allocates, so they call the entry point below instead.
 *
 * Its scratch is one file-scope device array of OFRL_NOALLOC_SCRATCH_BYTES,
 * reserved in every GPU that loads this library until the library is
 * unloaded.  The first call made with a given device current looks up the
 * array's device address (cudaGetSymbolAddress) and keeps it; make that first
 * call before any stream capture.  All calls share the one array: two calls
 * whose kernels overlap on the GPU (different streams, or different host
 * threads) race and give wrong results, so serialise them (one stream). */
#define OFRL_NOALLOC_SCRATCH_BYTES (4u << 20)

/* Largest batch ofrl_iql_value_fwd_bwd_noalloc accepts for `shape` (what the
 * scratch array holds), or -1 for an unsupported shape. */
int64_t ofrl_noalloc_max_batch(const ofrl_vshape* shape);

/* Same computation, arguments and results as ofrl_iql_value_fwd_bwd (V
 * forward, expectile loss, V backward into grad_out), with `shape` in place
 * of a context.  Allocates nothing: no cudaMalloc, no cudaFree, no allocating
 * library call.  A batch above ofrl_noalloc_max_batch(shape) returns
 * OFRL_EINVAL before anything is launched; H outside {64, 128, 256} returns
 * OFRL_EUNSUPPORTED.  Asynchronous on `stream`. */
ofrl_status ofrl_iql_value_fwd_bwd_noalloc(const ofrl_vshape* shape, const float* params, const float* states,
                                           int32_t state_stride, int32_t batch, const float* q_taken, float tau,
                                           float* v_out, float* loss_out, float* grad_out, void* stream);

/* ---- sequence memory: the gated delta rule over packed episodes ---------- */

/* A recurrent memory for states that are not Markov: an associative state
 * S [v_dim, k_dim] per value head, zero (or given) when an episode starts,
 *
 *   S_t = a_t S_{t-1} + u_t k_t^T,  a_t = exp(g_t),
 *   u_t = beta_t (v_t - a_t S_{t-1} k_t),   o_t = scale S_t q_t,
 *
 * so S_t k_t moves from its decayed prediction toward v_t by beta_t |k_t|^2.
 * With unit keys and beta in [0, 1] the state stays bounded.  g_t = -inf forgets
 * everything before t; g_t > 0, or beta |k|^2 above two, lets the state grow.
 * Where it grows by more than 2^16 within 64 tokens (2^24 with bf16 tokens and
 * no final_state) a forward call goes over the episode token by token, 1.5 to 3
 * microseconds each.  Beyond 2^20 (fp32 tokens) or 2^24 (bf16)
 * within 64 tokens, gradients of these tokens and of those before them in the
 * episode are NaN.  No counterpart on the pages, whose networks see one
 * transition at a time.
 *
 * What is kept of operands: fp32 tokens 22 bits and bf16 tokens 11, relative to
 * the largest element of a row of q or k, and of up to 64 tokens of v, states and
 * what is made of them; sums, decays and states are fp32, and with bf16 tokens
 * states asked for are made from 22 bits, d_init from 11.  Rows of k whose largest
 * element lies outside 2^-60 .. 2^60 keep fewer.
 *
 * Tokens are transitions in buffer order: token t of episode e lies between
 * episode_ends[e - 1] (0 for the first) and episode_ends[e], the convention of
 * ofrl_replay, except that an episode may be empty (its end repeats the one
 * before; its final state is its initial one).  The ends are device data: an
 * end below its predecessor or above `tokens` is counted in
 * OFRL_STAT_BAD_INDEX by the forward call, and what that call writes is then
 * unspecified (every access stays in bounds).  Tokens at and after the last
 * end belong to no episode; their outputs and gradients are not written.
 *
 * What is not finite stays where the recurrence takes it: an element of v in
 * its channel, k, g or beta of a token in all channels of the head, reach the
 * outputs and states from that token on, q its own output alone, and nothing
 * reaches an earlier token, another channel or another episode.  Gradients
 * keep to that for v; a q, k, g, beta or dout that is not finite may reach any
 * gradient of its episode.
 *
 * Value head h reads query and key head h / (v_heads / k_heads); dq and dk
 * sum over the value heads of a group, in a fixed order. */
enum { OFRL_DTYPE_F32 = 0, OFRL_DTYPE_BF16 = 1 };

typedef struct {
    int32_t k_heads;   /* query and key heads, 1 .. 1024 */
    int32_t v_heads;   /* value heads, a multiple of k_heads, at most 1024 */
    int32_t k_dim;     /* 8 .. 128, a multiple of 8 */
    int32_t v_dim;     /* 8 .. 128, a multiple of 8 */
    int32_t dtype;     /* OFRL_DTYPE_* of every token buffer (q k v g beta out and gradients); states are fp32 */
} ofrl_delta_shape;

/* Tokens of one call, device.  A stride is the distance between tokens in
 * elements; heads are contiguous within a token.  q, k, v: 16-byte aligned,
 * strides multiples of 16 bytes; g, beta: any stride >= v_heads. */
typedef struct {
    const void* q;       /* [tokens][k_heads, k_dim] */
    const void* k;       /* [tokens][k_heads, k_dim] */
    const void* v;       /* [tokens][v_heads, v_dim] */
    const void* g;       /* [tokens][v_heads] log decay */
    const void* beta;    /* [tokens][v_heads] write strength */
    int64_t q_stride, k_stride, v_stride, g_stride, beta_stride;
    int64_t tokens;      /* 0 .. 2^31-1 */
    float scale;         /* of the outputs, finite */
} ofrl_delta_tokens;

/* Gradients of one call, device, written (not accumulated): same layouts,
 * alignments and stride rules as the tokens they belong to. */
typedef struct {
    void* dq;
    void* dk;
    void* dv;
    void* dg;
    void* dbeta;
    int64_t q_stride, k_stride, v_stride, g_stride, beta_stride;
} ofrl_delta_grads;

typedef struct ofrl_delta ofrl_delta;

/* Create the workspace for sequences of up to max_tokens tokens in up to
 * max_episodes episodes (0 of each is enough for ofrl_delta_step alone;
 * backward = 0 reserves less and refuses ofrl_delta_backward).  The only
 * allocating call; binds to the current device.  One ofrl_delta must not be
 * used by two calls that overlap on the GPU. */
ofrl_status ofrl_delta_create(const ofrl_delta_shape* shape, int64_t max_tokens, int32_t max_episodes,
                              int32_t backward, ofrl_delta** out);
ofrl_status ofrl_delta_destroy(ofrl_delta* ctx);

/* As ofrl_poll_status, of the ofrl_delta's own status word. */
ofrl_status ofrl_delta_poll_status(ofrl_delta* ctx, void* stream, int32_t* words_out);

/* Bytes of device memory ofrl_delta_create reserves, or -1 for bad arguments. */
int64_t ofrl_delta_workspace_bytes(const ofrl_delta_shape* shape, int64_t max_tokens, int32_t max_episodes,
                                   int32_t backward);

/* Bytes of the `saved` buffer (device, 256-byte aligned, the caller's) that
 * hands a forward call's per-chunk states to its backward call, or -1. */
int64_t ofrl_delta_saved_bytes(const ofrl_delta_shape* shape, int64_t tokens, int32_t num_episodes);

/* Forward over packed episodes.  episode_ends: device [num_episodes].
 * init_state: device fp32 [num_episodes, v_heads, v_dim, k_dim], 16-byte
 * aligned, or NULL (zero).  out: device [tokens, v_heads, v_dim], contiguous,
 * 16-byte aligned.  final_state: as init_state, or NULL; may be init_state
 * (buffers that overlap otherwise are refused).
 * saved: device, ofrl_delta_saved_bytes, or NULL (no backward will follow). */
ofrl_status ofrl_delta_forward(ofrl_delta* ctx, const ofrl_delta_tokens* in, const int32_t* episode_ends,
                               int32_t num_episodes, const float* init_state, void* out, float* final_state,
                               void* saved, void* stream);

/* Backward of the forward call that filled `saved` with the same tokens and
 * ends: dout as `out`; d_final: gradient of final_state, fp32, or NULL (zero);
 * d_init: gradient of init_state, fp32, or NULL (not wanted); may be d_final
 * (buffers that overlap otherwise are refused). */
ofrl_status ofrl_delta_backward(ofrl_delta* ctx, const ofrl_delta_tokens* in, const int32_t* episode_ends,
                                int32_t num_episodes, const void* saved, const void* dout, const float* d_final,
                                const ofrl_delta_grads* grads, float* d_init, void* stream);

/* One token for each of in->tokens environments, each with a state of its
 * own: state_in, state_out device fp32 [slots, v_heads, v_dim, k_dim], 16-byte
 * aligned (the same buffer updates in place; buffers that overlap otherwise
 * are refused); slot_idx: device int32 [tokens], the state of each token, or
 * NULL (token i has state i, slots >= tokens).  Two tokens of one call must not name one slot.  A slot outside
 * [0, slots) is counted in OFRL_STAT_BAD_INDEX: its token's output is zero
 * and no state is written.  With slot_idx, slots of state_out that no token
 * names are left as they are. */
ofrl_status ofrl_delta_step(ofrl_delta* ctx, const ofrl_delta_tokens* in, const int32_t* slot_idx, int32_t slots,
                            const float* state_in, float* state_out, void* out, void* stream);

/* ---- state space blocks over packed episodes ------------------------------- */

/* The other sequence memory, and what stands around either one in a block:
 *
 *   short causal convolution    ofrl_conv_*       before the memory
 *   selective scan              ofrl_scan_*       the memory: decays per channel and state
 *   gated norm                  ofrl_gated_norm   after it
 *   residual norm               ofrl_residual_norm    before the next block
 *
 * Episodes are packed as for the gated delta rule: token t of episode e lies
 * between episode_ends[e - 1] (0 for the first) and episode_ends[e], device
 * int32, ascending, equal ends for an empty episode.  An end below its
 * predecessor or above `tokens` is counted in OFRL_STAT_BAD_INDEX by the
 * forward call, whose results are then unspecified (every access stays in
 * bounds).  Tokens at and after the last end belong to no episode; their
 * outputs and gradients are not written.
 *
 * Token buffers ("rows") have a stride, the distance between tokens in
 * elements, and contiguous elements within a token.  They are 16-byte aligned
 * with strides that are multiples of 16 bytes, except b and c of the scan,
 * which have any alignment and stride.  Token types are OFRL_DTYPE_*; weights,
 * their gradients, the scan's states and all arithmetic are fp32, and sums that
 * run over tokens are added in an order fixed by the sizes.  Outputs must not
 * overlap inputs unless said otherwise.  No counterpart on the pages, whose
 * networks see one transition at a time. */

/* out_t = act(bias + sum_{j < width} weight[j] x_{t - width + 1 + j}) per
 * channel, within an episode; before its first token stand the width - 1
 * inputs of init_state, oldest first, or zeros.  What is not finite stays in
 * its channel and in the `width` tokens from its own on. */
enum { OFRL_ACT_NONE = 0, OFRL_ACT_SILU = 1 };
typedef struct {
    int32_t channels;     /* 8 .. 65536, a multiple of 8 */
    int32_t width;        /* 2 .. 4 */
    int32_t activation;   /* OFRL_ACT_* */
    int32_t dtype;        /* OFRL_DTYPE_* of x, out, their gradients and the states */
} ofrl_conv_shape;

typedef struct {
    const void* x;          /* [tokens][channels] */
    const float* weight;    /* [channels, width] */
    const float* bias;      /* [channels] or NULL */
    int64_t x_stride;
    int64_t tokens;         /* 0 .. 2^31 - 2^17 */
} ofrl_conv_tokens;

/* Gradients, written (not accumulated). */
typedef struct {
    void* dx;               /* [tokens][channels] */
    float* dweight;         /* [channels, width] */
    float* dbias;           /* [channels] or NULL: not wanted */
    int64_t x_stride;
} ofrl_conv_grads;

typedef struct ofrl_conv ofrl_conv;

/* The workspace for calls of up to max_tokens tokens in up to max_episodes
 * episodes (0 of each is enough for ofrl_conv_step; backward = 0 refuses
 * ofrl_conv_backward).  The only allocating call; binds to the current device.
 * One ofrl_conv must not be used by two calls that overlap on the GPU. */
ofrl_status ofrl_conv_create(const ofrl_conv_shape* shape, int64_t max_tokens, int32_t max_episodes, int32_t backward,
                             ofrl_conv** out);
ofrl_status ofrl_conv_destroy(ofrl_conv* ctx);
ofrl_status ofrl_conv_poll_status(ofrl_conv* ctx, void* stream, int32_t* words_out);
int64_t ofrl_conv_workspace_bytes(const ofrl_conv_shape* shape, int64_t max_tokens, int32_t max_episodes,
                                  int32_t backward);

/* init_state, final_state: [num_episodes, channels, width - 1] in the tokens'
 * type, 16-byte aligned, or NULL (zeros; not wanted).  final_state holds each
 * episode's last width - 1 inputs (an episode of fewer ends on its initial
 * ones).  They must not overlap: parts of an episode run at the same time. */
ofrl_status ofrl_conv_forward(ofrl_conv* ctx, const ofrl_conv_tokens* in, const int32_t* episode_ends,
                              int32_t num_episodes, const void* init_state, void* out, int64_t out_stride,
                              void* final_state, void* stream);

/* Gradients of the forward call with the same inputs: dout rows of out's
 * gradient; d_final: gradient of final_state, in the tokens' type, or NULL;
 * d_init: gradient of init_state, fp32, or NULL (not wanted); it must not
 * overlap the other states. */
ofrl_status ofrl_conv_backward(ofrl_conv* ctx, const ofrl_conv_tokens* in, const int32_t* episode_ends,
                               int32_t num_episodes, const void* init_state, const void* dout, int64_t dout_stride,
                               const void* d_final, const ofrl_conv_grads* grads, float* d_init, void* stream);

/* One token for each of in->tokens environments: state_in, state_out [slots,
 * channels, width - 1] (the same buffer updates in place; buffers that overlap
 * otherwise are refused); slot_idx as ofrl_delta_step's. */
ofrl_status ofrl_conv_step(ofrl_conv* ctx, const ofrl_conv_tokens* in, const int32_t* slot_idx, int32_t slots,
                           const void* state_in, void* state_out, void* out, int64_t out_stride, void* stream);

/* Per channel d and state n, with B and C of the channel's group
 * (d / (channels / groups)):
 *
 *   delta_t = softplus(dt_t + dt_bias)           (or dt_t + dt_bias)
 *   h_t[n] = exp(delta_t A[n]) h_{t-1}[n] + delta_t B_t[n] x_t
 *   y_t = sum_n C_t[n] h_t[n] + D x_t,   out_t = y_t silu(z_t)   (z NULL: y_t)
 *
 * The state is zero, or init_state, when an episode starts.  What is not finite
 * stays where the recurrence takes it: x, dt and z of a channel in that
 * channel, B and C of a token in their group, from that token on and within
 * the episode.  Gradients keep to the episode, those of A, D and dt_bias,
 * which sum over tokens, excepted. */
typedef struct {
    int32_t channels;     /* 8 .. 65536 */
    int32_t state_dim;    /* N: 4 .. 64, a multiple of 4 */
    int32_t groups;       /* divides channels; channels / groups a multiple of 8 */
    int32_t dtype;        /* OFRL_DTYPE_* of every token buffer */
    int32_t softplus;     /* 1: delta = softplus(dt + dt_bias); 0: dt + dt_bias */
} ofrl_scan_shape;

typedef struct {
    const void* x;          /* [tokens][channels] */
    const void* dt;         /* [tokens][channels] */
    const void* b;          /* [tokens][groups, N] */
    const void* c;          /* [tokens][groups, N] */
    const void* z;          /* [tokens][channels] or NULL */
    const float* a;         /* [channels, N], 16-byte aligned; negative for states that decay */
    const float* d;         /* [channels] or NULL (zero) */
    const float* dt_bias;   /* [channels] or NULL (zero) */
    int64_t x_stride, dt_stride, b_stride, c_stride, z_stride;
    int64_t tokens;         /* 0 .. 2^31 - 2^17 */
} ofrl_scan_tokens;

/* Gradients, written (not accumulated); same layouts, alignments and stride
 * rules as what they belong to.  dz is NULL where z is; dd and ddt_bias may be
 * NULL (not wanted). */
typedef struct {
    void* dx;
    void* ddt;
    void* db;
    void* dc;
    void* dz;
    float* da;
    float* dd;
    float* ddt_bias;
    int64_t x_stride, dt_stride, b_stride, c_stride, z_stride;
} ofrl_scan_grads;

typedef struct ofrl_scan ofrl_scan;

/* As ofrl_conv_create and its companions. */
ofrl_status ofrl_scan_create(const ofrl_scan_shape* shape, int64_t max_tokens, int32_t max_episodes, int32_t backward,
                             ofrl_scan** out);
ofrl_status ofrl_scan_destroy(ofrl_scan* ctx);
ofrl_status ofrl_scan_poll_status(ofrl_scan* ctx, void* stream, int32_t* words_out);
int64_t ofrl_scan_workspace_bytes(const ofrl_scan_shape* shape, int64_t max_tokens, int32_t max_episodes,
                                  int32_t backward);

/* Bytes of the `saved` buffer (device, 16-byte aligned, the caller's) that
 * hands a forward call's states to its backward call, or -1. */
int64_t ofrl_scan_saved_bytes(const ofrl_scan_shape* shape, int64_t tokens);

/* init_state, final_state: device fp32 [num_episodes, channels, N], 16-byte
 * aligned, or NULL (zero; not wanted).  They must not overlap: parts of an
 * episode run at the same time.  saved: as above, or NULL (no backward call will follow). */
ofrl_status ofrl_scan_forward(ofrl_scan* ctx, const ofrl_scan_tokens* in, const int32_t* episode_ends,
                              int32_t num_episodes, const float* init_state, void* out, int64_t out_stride,
                              float* final_state, void* saved, void* stream);

/* Gradients of the forward call that filled `saved` with the same inputs: dout
 * rows of out's gradient; d_final: gradient of final_state, or NULL (zero);
 * d_init: gradient of init_state, or NULL (not wanted); it must not overlap the
 * other states. */
ofrl_status ofrl_scan_backward(ofrl_scan* ctx, const ofrl_scan_tokens* in, const int32_t* episode_ends,
                               int32_t num_episodes, const float* init_state, const void* saved, const void* dout,
                               int64_t dout_stride, const float* d_final, const ofrl_scan_grads* grads, float* d_init,
                               void* stream);

/* One token for each of in->tokens environments: state_in, state_out fp32
 * [slots, channels, N], 16-byte aligned (the same buffer updates in place;
 * buffers that overlap otherwise are refused); slot_idx as ofrl_delta_step's. */
ofrl_status ofrl_scan_step(ofrl_scan* ctx, const ofrl_scan_tokens* in, const int32_t* slot_idx, int32_t slots,
                           const float* state_in, float* state_out, void* out, int64_t out_stride, void* stream);

/* Norms of rows: rms(v) = sqrt(mean(v^2) + eps) over each of `groups` equal
 * groups of a row's channels.
 *
 *   gated norm      gate_first = 0:  out = weight x / rms(x) silu(z)
 *                   gate_first = 1:  out = weight u / rms(u),  u = x silu(z)
 *   residual norm   h = residual + scale x,  residual_out = h,  out = weight h / rms(h)
 *
 * A row is read whole before its outputs are written, so in a forward call out
 * may be x (same stride), and residual_out may be residual where no backward
 * call follows.  What is not finite stays in its row and group (and in the
 * sums over rows that are the weights' gradients).  Squares are summed in fp32 as
 * they are: values from about 1e18 on have an infinite rms. */
typedef struct {
    int32_t channels;        /* 8 .. 65536 */
    int32_t groups;          /* divides channels; channels / groups a multiple of 8, at most 8192 */
    int32_t dtype;           /* OFRL_DTYPE_* of x, z, out and their gradients */
    int32_t residual_dtype;  /* of residual, residual_out and their gradients: OFRL_DTYPE_F32 or dtype */
} ofrl_norm_shape;

typedef struct {
    const void* x;           /* [rows][channels] */
    const void* z;           /* [rows][channels] */
    const float* weight;     /* [channels], 16-byte aligned */
    int64_t x_stride, z_stride;
    int64_t rows;            /* 0 .. 2^31-1 */
    float eps;               /* > 0, finite */
    int32_t gate_first;
} ofrl_gated_rows;

typedef struct {
    const void* x;           /* [rows][channels] */
    const void* residual;    /* [rows][channels] */
    const float* scale;      /* [channels], 16-byte aligned, or NULL (one) */
    const float* weight;     /* [channels], 16-byte aligned */
    int64_t x_stride, residual_stride;
    int64_t rows;
    float eps;
} ofrl_residual_rows;

typedef struct ofrl_norm ofrl_norm;

/* The workspace (its size does not depend on the rows; backward = 0 refuses the
 * backward calls).  The only allocating call; binds to the current device.
 * Backward calls keep their parts of the weights' gradients in it: one ofrl_norm
 * must not be used by two of them that overlap on the GPU.  Forward calls use
 * none of it. */
ofrl_status ofrl_norm_create(const ofrl_norm_shape* shape, int32_t backward, ofrl_norm** out);
ofrl_status ofrl_norm_destroy(ofrl_norm* ctx);
int64_t ofrl_norm_workspace_bytes(const ofrl_norm_shape* shape, int32_t backward);

ofrl_status ofrl_gated_norm(ofrl_norm* ctx, const ofrl_gated_rows* in, void* out, int64_t out_stride, void* stream);

/* dx, dz rows, dweight fp32 [channels], written (not accumulated); dx may be
 * dout and dz may be z (same strides). */
ofrl_status ofrl_gated_norm_backward(ofrl_norm* ctx, const ofrl_gated_rows* in, const void* dout, int64_t dout_stride,
                                     void* dx, int64_t dx_stride, void* dz, int64_t dz_stride, float* dweight,
                                     void* stream);

ofrl_status ofrl_residual_norm(ofrl_norm* ctx, const ofrl_residual_rows* in, void* residual_out,
                               int64_t residual_out_stride, void* out, int64_t out_stride, void* stream);

/* d_residual_out: gradient of residual_out, or NULL (zero).  dx; dresidual, in
 * the residual's type; dweight and dscale (NULL where scale is) fp32
 * [channels]; written (not accumulated).  dx may be dout and dresidual may be
 * d_residual_out (same strides). */
ofrl_status ofrl_residual_norm_backward(ofrl_norm* ctx, const ofrl_residual_rows* in, const void* dout,
                                        int64_t dout_stride, const void* d_residual_out, int64_t d_residual_out_stride,
                                        void* dx, int64_t dx_stride, void* dresidual, int64_t dresidual_stride,
                                        float* dweight, float* dscale, void* stream);

/* ---- gradients kept in many tensors ---------------------------------------- */

/* A list of n device tensors (host arrays of pointers, element counts and
 * OFRL_DTYPE_* types; a size may be 0 and its pointer then NULL; pointers
 * aligned to their element; n 1 .. 2^20).  Creating it copies the list to the
 * device (the only allocation; the scratch of the calls below is part of it);
 * the tensors stay the caller's and must outlive it.  One list must not be
 * used by two calls that overlap on the GPU. */
typedef struct ofrl_tensors ofrl_tensors;
ofrl_status ofrl_tensors_create(const void* const* ptrs, const int64_t* sizes, const int32_t* dtypes, int32_t n,
                                ofrl_tensors** out);
ofrl_status ofrl_tensors_destroy(ofrl_tensors* list);

/* norm_out[0] (device fp32) = the 2-norm over all elements of all tensors:
 * fp32 squares summed in a fixed order.  Next to ofrl_adam_step, whose
 * grad_norm it is: each parameter tensor's step then clips by the global
 * norm.  Non-finite elements make it non-finite. */
ofrl_status ofrl_global_norm(ofrl_tensors* list, float* norm_out, void* stream);

/* The norm n as above, then every element times s = (n > max_norm && n > 0)
 * ? max_norm / n : 1 ("DQN Backward-Path NaN Audit", the clip formula),
 * rounded to its tensor's type.  out: a list with the same sizes and types
 * that receives the result (it must not overlap `list`), or NULL: in place.
 * max_norm > 0 (+inf: s = 1). */
ofrl_status ofrl_global_norm_clip(ofrl_tensors* list, float max_norm, float* norm_out, ofrl_tensors* out,
                                  void* stream);

/* ---- measurement hooks (not part of the method) ----------------------- */

/* Phases of ofrl_train_step, in launch order. */
enum { OFRL_PHASE_RELABEL = 0, OFRL_PHASE_VNET = 1, OFRL_PHASE_REDUCE = 2, OFRL_PHASE_ADAM = 3,
       OFRL_PHASES = 4 };

/* Start recording per-phase device time of the next max_steps calls of
 * ofrl_train_step on this context: CUDA events recorded on the call's stream
 * around each phase (host-side event objects are created here; no device
 * memory is allocated).  A second begin replaces the first. */
ofrl_status ofrl_profile_begin(ofrl_ctx* ctx, int32_t max_steps);

/* Wait for the recorded events, write the summed time of each phase in
 * milliseconds to phase_ms_out[OFRL_PHASES] and the number of recorded steps
 * to *steps_out, and stop recording. */
ofrl_status ofrl_profile_end(ofrl_ctx* ctx, float* phase_ms_out, int32_t* steps_out);

#ifdef __cplusplus
}
#endif
#endif /* OFRL_H */
