// Gated delta rule over packed episodes, forward and backward, by chunks of
// 64 tokens.  With G_i the running sum of log decays inside a chunk, gamma_i
// = exp(G_i), D_ij = exp(G_i - G_j) for j <= i, S_0 the state before it and
// S_1 the one after, row vectors per token:
//   x_i = v_i - gamma_i S_0 k_i
//   (1 + A) u = beta x,   A_ij = beta_i D_ij (k_i k_j), j < i
//   o_i = scale (gamma_i S_0 q_i + sum_{j<=i} P_ij u_j),   P_ij = D_ij (q_i k_j)
//   S_1 = gamma_last S_0 + sum_j exp(G_last - G_j) u_j k_j^T
// and backward, with T = (1 + A)^-1:
//   du = scale P^T do + exp(G_last - G_j) dS_1 k_j,   r = T^T du,   dv = beta r
//   dS_0 = gamma_last dS_1 + scale sum gamma_i do_i q_i^T - sum gamma_i dv_i k_i^T
//   dP = scale do u^T,  dA = -r u^T,  M_ij = beta_i dA_ij D_ij
//   dq_i = scale gamma_i S_0^T do_i + sum_j dP_ij D_ij k_j
//   dk_i = [-gamma_i S_0^T dv_i + sum_j M_ij k_j]                        (row part)
//        + [sum_m dP_mi D_mi q_m + sum_m M_mi k_m + exp(G_last - G_i) dS_1^T u_i]   (column part)
//   dbeta_i = r_i x_i + sum_j dA_ij D_ij (k_i k_j)
//   dG_i = q_i (state part of dq_i) + k_i (state part of the row part) - k_i (state part of the column part)
//        + sum_j N_ij - sum_m N_mi,   N = dP P + dA A   (and more at the last token)
//   dg_i = sum_{m >= i} dG_m = <S_0, dS_0> - sum_{m < i} dG_m,
//   <S_0, dS_0> = gamma_last <S_0, dS_1> + sum_i [q_i (state part of dq_i) + k_i (state part of the row part)]:
// S_0 enters times exp(G) only.  The second form of dg_i is taken: it is exactly zero where S_0 is.
//
// Read: one launch where token by token is taken (delta_step.cu), else two, or
// four in parts (delta_chain.cu).  Learn: two forward and two back.
// delta_prep.cu makes per chunk what needs no state (T, P, scaled keys and
// queries); delta_chain.cu and delta_chain_tc.cu walk the chunks of every episode
// forward and, for gradients, back; delta_grad.cu and delta_grad_tc.cu then take
// every chunk by itself; delta_redo.cuh goes over an episode whose states do not
// stay finite or within the chunks' range.  This file lays out the buffers between
// them.

#include <algorithm>

#include "delta_mma.cuh"

namespace ofrl {
namespace delta {
namespace {

inline int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

struct Sizes {
    int64_t keys, pairs, state, vec, units;
};
Sizes sizes_of(const ofrl_delta_shape& s, int64_t slots) {
    const int planes = token_planes(s.dtype), dk = pad_dim(s.k_dim), dv = pad_dim(s.v_dim);
    Sizes z;
    z.keys = round_up(slots * s.k_heads * KeyImage::bytes(dk, planes), 256);
    z.pairs = round_up(slots * s.v_heads * kPairBytes, 256);
    z.state = round_up(slots * s.v_heads * planes * dv * dk * 2, 256);
    z.vec = round_up(slots * s.v_heads * planes * dv * kChunk * 2, 256);
    z.units = round_up(slots * s.v_heads * 4, 256);
    return z;
}

Prepared prepared_at(uint8_t* p, const Sizes& z) { return {p, p + z.keys}; }
Images images_at(uint8_t* p, const Sizes& z) {
    return {p, p + z.state, reinterpret_cast<float*>(p + z.state + z.vec),
            reinterpret_cast<float*>(p + z.state + z.vec + z.units)};
}
int64_t prepared_bytes(const Sizes& z) { return z.keys + z.pairs; }
int64_t images_bytes(const Sizes& z) { return z.state + z.vec + 2 * z.units; }

// bf16 outputs need 11 significand bits of every operand, fp32 outputs 22;
// final states are fp32 whatever the tokens are.
int planes_of(const SeqLaunch& a) { return a.shape.dtype == OFRL_DTYPE_F32 || a.final_state ? 2 : 1; }

// Whether token by token is the faster way, by estimates of both in us.  Token
// by token: a step of an episode takes 0.28 us, a CTA costs 3.7 ns of the whole
// GPU's time to start and 32 lanes' share of a token 0.11 ns.  Chunked: 10.4 us
// for two launches and one chunk (13.8 with two planes), then 25 ns for each
// chunk of a head, times the planes, twice for more than 64 channels.  The host
// knows the mean length only and takes the longest episode for twice that; the
// bound on the tokens keeps the worst case, all of them in one episode, at 2 ms
// (one episode of 3801 tokens among 199 of one, one head of 64, fp32: 1100 us,
// chunked 298; one of 7600 among 399, 8 x 8: 1774 and 588).
// Measured, two heads of 64, fp32, token by token / chunked: 16 episodes of 16
// tokens 7.2 / 13.8 us, of 48 16.4 / 14.6; 1024 of 4 47.7 / 129.7; 256 of 32
// 68.7 / 40.2.  Four heads of 128, bf16: 16 of 4 7.8 / 13.3, 64 of 16 68.9 / 22.2.
bool recurrent(const SeqLaunch& a) {
    if (a.in.tokens > 8192) return false;
    const int lanes = a.shape.k_dim > 64 ? 32 : a.shape.k_dim > 32 ? 16 : 8;
    const int rows = recur_rows(lanes), planes = planes_of(a);
    const double heads = (double)a.episodes * a.shape.v_heads, length = (double)a.in.tokens / a.episodes;
    const double ctas = heads * ((a.shape.v_dim + rows - 1) / rows);
    const double token = 2.7 + std::max(0.28 * 2 * length, 0.0037 * ctas + 1.1e-4 * heads * length * a.shape.v_dim * lanes / 32);
    const double chunks = heads * std::max(1.0, length / kChunk);
    const bool wide = a.shape.k_dim > 64 || a.shape.v_dim > 64;
    return token < (planes == 2 ? 13.8 : 10.4) + 0.025 * chunks * planes * (wide ? 2 : 1);
}

}  // namespace

// What a forward call without `saved` needs, or a backward call, whichever is more.
int64_t scratch_bytes(const ofrl_delta_shape& s, int64_t tokens, int64_t episodes, bool backward) {
    const Sizes z = sizes_of(s, slots_of(tokens, episodes));
    const int64_t f = prepared_bytes(z), b = backward ? images_bytes(z) : 0;
    return f > b ? f : b;
}

// Room for the parts of a forward pass: segments_of() makes no more of them
// than the SMs hold CTAs, two each.
int64_t parts_bytes(const ofrl_delta_shape& s, int64_t tokens, int num_sms) {
    if (tokens < 12 * kChunk) return 0;
    const int64_t dk = pad_dim(s.k_dim);
    return 3LL * num_sms * (s.v_dim * s.k_dim * 4 + 4 * dk * dk + 32) + 256;
}

int64_t saved_bytes(const ofrl_delta_shape& s, int64_t tokens, int64_t episodes) {
    const Sizes z = sizes_of(s, slots_of(tokens, episodes));
    return prepared_bytes(z) + images_bytes(z);
}

cudaError_t launch_forward(const SeqLaunch& a, cudaStream_t st) {
    if (!a.saved && recurrent(a)) return launch_recur(a, st);
    const Sizes z = sizes_of(a.shape, slots_of(a.in.tokens, a.episodes));
    const Prepared p = prepared_at(a.saved ? a.saved : a.scratch, z);
    Images img = {};
    if (a.saved) img = images_at(a.saved + prepared_bytes(z), z);
    const int planes = planes_of(a);
    const cudaError_t e = launch_prep(a, p, planes, st);
    return e == cudaSuccess ? launch_chain_forward(a, p, img, planes, st) : e;
}

cudaError_t launch_backward(const SeqLaunch& a, cudaStream_t st) {
    const Sizes z = sizes_of(a.shape, slots_of(a.in.tokens, a.episodes));
    const Prepared p = prepared_at(a.saved, z);
    const Images fwd = images_at(a.saved + prepared_bytes(z), z), rev = images_at(a.scratch, z);
    const cudaError_t e = launch_chain_reverse(a, p, rev, st);
    if (e != cudaSuccess) return e;
    return a.shape.dtype == OFRL_DTYPE_F32 ? launch_grad(a, p, fwd, rev, st) : launch_grad_tc(a, p, fwd, rev, st);
}

}  // namespace delta
}  // namespace ofrl
