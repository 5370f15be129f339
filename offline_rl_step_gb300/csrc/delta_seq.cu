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
// This file holds them as they stand: one CTA per (episode, key head) and
// plain loops in fp32 over work arrays in global memory.

#include "delta.cuh"

namespace ofrl {
namespace delta {
namespace {

constexpr int kThreads = 256;
constexpr int C = kChunk;
constexpr int kCtasPerSm = 2;

struct Scratch {
    float *S, *dS, *dSn, *KK, *A, *Ti, *P, *dP, *dA, *X, *U, *dU, *R, *vec;
};
__host__ __device__ inline int64_t scratch_floats(int dk, int dv) {
    return 3 * (int64_t)dk * dv + 6 * C * C + 4 * (int64_t)C * dv + 16 * C;
}
__device__ inline Scratch carve(float* p, int dk, int dv) {
    Scratch s;
    auto take = [&](int64_t n) { float* at = p; p += n; return at; };
    s.S = take((int64_t)dk * dv);
    s.dS = take((int64_t)dk * dv);
    s.dSn = take((int64_t)dk * dv);
    s.KK = take(C * C);
    s.A = take(C * C);
    s.Ti = take(C * C);
    s.P = take(C * C);
    s.dP = take(C * C);
    s.dA = take(C * C);
    s.X = take((int64_t)C * dv);
    s.U = take((int64_t)C * dv);
    s.dU = take((int64_t)C * dv);
    s.R = take((int64_t)C * dv);
    s.vec = take(16 * C);
    return s;
}

// Tokens of one chunk as functions of (row, channel); rows past the chunk are zero.
template <typename T>
struct ChunkTokens {
    const T *q, *k, *v, *g, *b;
    int64_t qs, ks, vs, gs, bs;
    int rows;
    __device__ float Q(int i, int c) const { return i < rows ? to_f(q[i * qs + c]) : 0.0f; }
    __device__ float K(int i, int c) const { return i < rows ? to_f(k[i * ks + c]) : 0.0f; }
    __device__ float V(int i, int c) const { return i < rows ? to_f(v[i * vs + c]) : 0.0f; }
    __device__ float G(int i) const { return i < rows ? fmaxf(to_f(g[i * gs]), kMinLogDecay) : 0.0f; }
    __device__ float B(int i) const { return i < rows ? to_f(b[i * bs]) : 0.0f; }
};

template <typename T>
__device__ ChunkTokens<T> chunk_tokens(const SeqLaunch& a, int64_t tok, int rows, int khead, int head) {
    ChunkTokens<T> t;
    t.q = static_cast<const T*>(a.in.q) + tok * a.in.q_stride + (int64_t)khead * a.shape.k_dim;
    t.k = static_cast<const T*>(a.in.k) + tok * a.in.k_stride + (int64_t)khead * a.shape.k_dim;
    t.v = static_cast<const T*>(a.in.v) + tok * a.in.v_stride + (int64_t)head * a.shape.v_dim;
    t.g = static_cast<const T*>(a.in.g) + tok * a.in.g_stride + head;
    t.b = static_cast<const T*>(a.in.beta) + tok * a.in.beta_stride + head;
    t.qs = a.in.q_stride;
    t.ks = a.in.k_stride;
    t.vs = a.in.v_stride;
    t.gs = a.in.g_stride;
    t.bs = a.in.beta_stride;
    t.rows = rows;
    return t;
}

// out(i, j, sum_k f(i, j, k)) over an m x n grid, then a block barrier.
template <typename F, typename O>
__device__ void mm(int m, int n, int k, F f, O out) {
    for (int x = threadIdx.x; x < m * n; x += kThreads) {
        const int i = x / n, j = x % n;
        float s = 0.0f;
        for (int c = 0; c < k; ++c) s += f(i, j, c);
        out(i, j, s);
    }
    __syncthreads();
}

// Decays, KK, A, T, P, X and U of a chunk, from S.  vec: G, gamma, rest, beta.
template <typename T>
__device__ void chunk_forward(const Scratch& w, const ChunkTokens<T>& t, int dk, int dv) {
    float *G = w.vec, *gam = w.vec + C, *rest = w.vec + 2 * C, *beta = w.vec + 3 * C;
    if (threadIdx.x == 0) {
        double sum = 0.0;
        for (int i = 0; i < C; ++i) G[i] = (float)(sum += t.G(i));
    }
    __syncthreads();
    for (int i = threadIdx.x; i < C; i += kThreads) {
        gam[i] = expf(G[i]);
        rest[i] = expf(G[C - 1] - G[i]);
        beta[i] = t.B(i);
    }
    __syncthreads();
    auto decay = [&](int i, int j) { return expf(G[i] - G[j]); };
    mm(C, C, dk, [&](int i, int j, int c) { return j < i ? t.K(i, c) * t.K(j, c) : 0.0f; },
       [&](int i, int j, float s) {
           w.KK[i * C + j] = j < i ? s * decay(i, j) : 0.0f;
           w.A[i * C + j] = j < i ? beta[i] * s * decay(i, j) : 0.0f;
       });
    mm(C, C, dk, [&](int i, int j, int c) { return j <= i ? t.Q(i, c) * t.K(j, c) : 0.0f; },
       [&](int i, int j, float s) { w.P[i * C + j] = j <= i ? s * decay(i, j) : 0.0f; });
    for (int j = threadIdx.x; j < C; j += kThreads)   // one column of (1 + A)^-1 per thread
        for (int i = 0; i < C; ++i) {
            float s = i == j ? 1.0f : 0.0f;
            for (int m = j; m < i; ++m) s -= w.A[i * C + m] * w.Ti[m * C + j];
            w.Ti[i * C + j] = i < j ? 0.0f : s;
        }
    mm(C, dv, dk, [&](int i, int v, int c) { return w.S[v * dk + c] * t.K(i, c); },
       [&](int i, int v, float s) { w.X[i * dv + v] = t.V(i, v) - gam[i] * s; });
    mm(C, dv, C, [&](int i, int v, int j) { return j <= i ? w.Ti[i * C + j] * beta[j] * w.X[j * dv + v] : 0.0f; },
       [&](int i, int v, float s) { w.U[i * dv + v] = s; });
}

template <typename T>
__global__ void __launch_bounds__(kThreads) delta_forward_simple(const __grid_constant__ SeqLaunch a) {
    const int dk = a.shape.k_dim, dv = a.shape.v_dim, hv = a.shape.v_heads, group = hv / a.shape.k_heads;
    const int64_t states = (int64_t)dk * dv;
    const Scratch w = carve(a.scratch + blockIdx.x * scratch_floats(dk, dv), dk, dv);
    for (int64_t item = blockIdx.x; item < (int64_t)a.episodes * hv; item += gridDim.x) {
        const int e = (int)(item / hv), head = (int)(item % hv), khead = head / group;
        const Span sp = span_of(a.ends, e, (int32_t)a.in.tokens);
        if (threadIdx.x == 0 && head == 0 && span_bad(a.ends, e, (int32_t)a.in.tokens))
            atomicAdd(a.status + OFRL_STAT_BAD_INDEX, 1);
        for (int64_t x = threadIdx.x; x < states; x += kThreads)
            w.S[x] = a.init ? a.init[((int64_t)e * hv + head) * states + x] : 0.0f;
        __syncthreads();
        for (int c0 = 0; c0 < sp.len; c0 += C) {
            const int64_t tok = (int64_t)sp.start + c0;
            if (a.saved) {
                float* to = reinterpret_cast<float*>(a.saved) +
                            (((int64_t)sp.start / C + e + c0 / C) * hv + head) * states;
                for (int64_t x = threadIdx.x; x < states; x += kThreads) to[x] = w.S[x];
            }
            const ChunkTokens<T> t = chunk_tokens<T>(a, tok, min(C, sp.len - c0), khead, head);
            chunk_forward(w, t, dk, dv);
            const float *gam = w.vec + C, *rest = w.vec + 2 * C;
            T* out = static_cast<T*>(a.out);
            mm(t.rows, dv, dk + C,
               [&](int i, int v, int c) {
                   return c < dk ? gam[i] * w.S[v * dk + c] * t.Q(i, c) : w.P[i * C + c - dk] * w.U[(c - dk) * dv + v];
               },
               [&](int i, int v, float s) { out[((tok + i) * hv + head) * dv + v] = from_f<T>(a.in.scale * s); });
            mm(dv, dk, C, [&](int v, int c, int j) { return rest[j] * w.U[j * dv + v] * t.K(j, c); },
               [&](int v, int c, float s) { w.S[v * dk + c] = gam[C - 1] * w.S[v * dk + c] + s; });
        }
        if (a.final_state)
            for (int64_t x = threadIdx.x; x < states; x += kThreads)
                a.final_state[((int64_t)e * hv + head) * states + x] = w.S[x];
        __syncthreads();
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) delta_backward_simple(const __grid_constant__ SeqLaunch a) {
    const int dk = a.shape.k_dim, dv = a.shape.v_dim, hv = a.shape.v_heads, hk = a.shape.k_heads, group = hv / hk;
    const int64_t states = (int64_t)dk * dv;
    const Scratch w = carve(a.scratch + blockIdx.x * scratch_floats(dk, dv), dk, dv);
    float *gam = w.vec + C, *rest = w.vec + 2 * C, *beta = w.vec + 3 * C;
    float *dG = w.vec + 4 * C, *db = w.vec + 5 * C, *rowdot = w.vec + 6 * C, *part = w.vec + 7 * C;
    const float scale = a.in.scale;
    for (int64_t item = blockIdx.x; item < (int64_t)a.episodes * hk; item += gridDim.x) {
        const int e = (int)(item / hk), khead = (int)(item % hk);
        const Span sp = span_of(a.ends, e, (int32_t)a.in.tokens);
        for (int head = khead * group; head < (khead + 1) * group; ++head) {
            const bool first = head == khead * group, last = head == (khead + 1) * group - 1;
            for (int64_t x = threadIdx.x; x < states; x += kThreads)
                w.dS[x] = a.d_final ? a.d_final[((int64_t)e * hv + head) * states + x] : 0.0f;
            __syncthreads();
            for (int c0 = (sp.len - 1) / C * C; sp.len > 0 && c0 >= 0; c0 -= C) {
                const int64_t tok = (int64_t)sp.start + c0;
                const float* from = reinterpret_cast<const float*>(a.saved) +
                                    (((int64_t)sp.start / C + e + c0 / C) * hv + head) * states;
                for (int64_t x = threadIdx.x; x < states; x += kThreads) w.S[x] = from[x];
                __syncthreads();
                const ChunkTokens<T> t = chunk_tokens<T>(a, tok, min(C, sp.len - c0), khead, head);
                chunk_forward(w, t, dk, dv);
                const T* dop = static_cast<const T*>(a.dout) + (tok * hv + head) * dv;
                auto dO = [&](int i, int v) { return i < t.rows ? to_f(dop[(int64_t)i * hv * dv + v]) : 0.0f; };
                auto decay = [&](int i, int j) { return expf(w.vec[i] - w.vec[j]); };
                mm(C, dv, C + dk,
                   [&](int j, int v, int c) {
                       return c < C ? scale * w.P[c * C + j] * dO(c, v) : rest[j] * w.dS[v * dk + c - C] * t.K(j, c - C);
                   },
                   [&](int j, int v, float s) { w.dU[j * dv + v] = s; });
                mm(C, dv, C, [&](int j, int v, int i) { return i >= j ? w.Ti[i * C + j] * w.dU[i * dv + v] : 0.0f; },
                   [&](int j, int v, float s) {
                       w.R[j * dv + v] = s;
                       if (j < t.rows)
                           static_cast<T*>(a.grads.dv)[(tok + j) * a.grads.v_stride + (int64_t)head * dv + v] =
                               from_f<T>(beta[j] * s);
                   });
                mm(C, C, dv, [&](int i, int j, int v) { return j <= i ? scale * dO(i, v) * w.U[j * dv + v] : 0.0f; },
                   [&](int i, int j, float s) { w.dP[i * C + j] = s; });
                mm(C, C, dv, [&](int i, int j, int v) { return j < i ? -w.R[i * dv + v] * w.U[j * dv + v] : 0.0f; },
                   [&](int i, int j, float s) { w.dA[i * C + j] = s; });
                mm(C, 1, C + dv,
                   [&](int i, int, int j) {
                       return j < C ? w.dA[i * C + j] * w.KK[i * C + j] : w.R[i * dv + j - C] * w.X[i * dv + j - C];
                   },
                   [&](int i, int, float s) { db[i] = s; });
                mm(C, 1, C,
                   [&](int i, int, int j) {
                       return w.dP[i * C + j] * w.P[i * C + j] + w.dA[i * C + j] * w.A[i * C + j] -
                              w.dP[j * C + i] * w.P[j * C + i] - w.dA[j * C + i] * w.A[j * C + i];
                   },
                   [&](int i, int, float s) { dG[i] = s; });
                // state parts and their row dots: one row per thread
                float* acc = a.grad_acc;
                const int64_t row_floats = (int64_t)hk * dk;
                for (int i = threadIdx.x; i < t.rows; i += kThreads) {
                    float* aq = acc + (tok + i) * 2 * row_floats + (int64_t)khead * dk;
                    float* ak = aq + row_floats;
                    float dots = 0.0f, col = 0.0f;
                    for (int c = 0; c < dk; ++c) {
                        float sq = 0.0f, sk = 0.0f, sc = 0.0f;
                        for (int v = 0; v < dv; ++v) {
                            sq += w.S[v * dk + c] * dO(i, v);
                            sk += w.S[v * dk + c] * w.R[i * dv + v];
                            sc += w.dS[v * dk + c] * w.U[i * dv + v];
                        }
                        sq *= scale * gam[i];
                        sk *= -gam[i] * beta[i];
                        sc *= rest[i];
                        dots += t.Q(i, c) * sq + t.K(i, c) * sk;
                        col += t.K(i, c) * sc;
                        float q = sq, k = sk + sc;
                        for (int j = 0; j < t.rows; ++j) {
                            if (j <= i) q += w.dP[i * C + j] * decay(i, j) * t.K(j, c);
                            if (j < i) k += beta[i] * w.dA[i * C + j] * decay(i, j) * t.K(j, c);
                            if (j >= i) k += w.dP[j * C + i] * decay(j, i) * t.Q(j, c);
                            if (j > i) k += beta[j] * w.dA[j * C + i] * decay(j, i) * t.K(j, c);
                        }
                        q += first ? 0.0f : aq[c];
                        k += first ? 0.0f : ak[c];
                        aq[c] = q;
                        ak[c] = k;
                        if (last) {
                            static_cast<T*>(a.grads.dq)[(tok + i) * a.grads.q_stride + (int64_t)khead * dk + c] =
                                from_f<T>(q);
                            static_cast<T*>(a.grads.dk)[(tok + i) * a.grads.k_stride + (int64_t)khead * dk + c] =
                                from_f<T>(k);
                        }
                    }
                    dG[i] += dots - col;
                    rowdot[i] = dots;
                }
                __syncthreads();
                mm(4 * C, 1, (int)((states + 4 * C - 1) / (4 * C)),
                   [&](int p, int, int n) {
                       const int64_t x = (int64_t)n * 4 * C + p;
                       return x < states ? w.S[x] * w.dS[x] : 0.0f;
                   },
                   [&](int p, int, float s) { part[p] = s; });
                if (threadIdx.x == 0) {
                    double sum = 0.0;
                    for (int p = 0; p < 4 * C; ++p) sum += (double)gam[C - 1] * part[p];
                    for (int i = 0; i < t.rows; ++i) sum += rowdot[i];
                    for (int i = 0; i < t.rows; ++i) {
                        static_cast<T*>(a.grads.dg)[(tok + i) * a.grads.g_stride + head] = from_f<T>((float)sum);
                        static_cast<T*>(a.grads.dbeta)[(tok + i) * a.grads.beta_stride + head] = from_f<T>(db[i]);
                        sum -= dG[i];
                    }
                }
                __syncthreads();
                mm(dv, dk, C,
                   [&](int v, int c, int i) {
                       return gam[i] * (scale * dO(i, v) * t.Q(i, c) - beta[i] * w.R[i * dv + v] * t.K(i, c));
                   },
                   [&](int v, int c, float s) { w.dSn[v * dk + c] = gam[C - 1] * w.dS[v * dk + c] + s; });
                for (int64_t x = threadIdx.x; x < states; x += kThreads) w.dS[x] = w.dSn[x];
                __syncthreads();
            }
            if (a.d_init)
                for (int64_t x = threadIdx.x; x < states; x += kThreads)
                    a.d_init[((int64_t)e * hv + head) * states + x] = w.dS[x];
            __syncthreads();
        }
    }
}

int grid_for(const SeqLaunch& a, int64_t items) {
    const int64_t most = (int64_t)a.num_sms * kCtasPerSm;
    return (int)(items < most ? items : most);
}

}  // namespace

int64_t scratch_bytes(const ofrl_delta_shape& s, int num_sms) {
    return (int64_t)num_sms * kCtasPerSm * scratch_floats(s.k_dim, s.v_dim) * 4;
}

int64_t saved_bytes(const ofrl_delta_shape& s, int64_t tokens, int64_t episodes) {
    return slots_of(tokens, episodes) * s.v_heads * s.k_dim * s.v_dim * 4;
}

cudaError_t launch_forward(const SeqLaunch& a, cudaStream_t st) {
    const int grid = grid_for(a, (int64_t)a.episodes * a.shape.v_heads);
    if (a.shape.dtype == OFRL_DTYPE_F32)
        delta_forward_simple<float><<<grid, kThreads, 0, st>>>(a);
    else
        delta_forward_simple<__nv_bfloat16><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_backward(const SeqLaunch& a, cudaStream_t st) {
    const int grid = grid_for(a, (int64_t)a.episodes * a.shape.k_heads);
    if (a.shape.dtype == OFRL_DTYPE_F32)
        delta_backward_simple<float><<<grid, kThreads, 0, st>>>(a);
    else
        delta_backward_simple<__nv_bfloat16><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace delta
}  // namespace ofrl
