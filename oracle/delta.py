"""Gated delta rule, token by token in fp64: forward, adjoint and one step (numpy).

Per value head, S [v_dim, k_dim] starts at zero or at the given state and
    old = exp(g) S,  err = v - old k,  u = beta err,  S = old + u k^T,  o = scale S q.
Value head h reads key head h // (v_heads // k_heads).
"""
import numpy as np


def _spans(ends):
    start = 0
    for e in ends:
        yield start, int(e)
        start = int(e)


def forward(q, k, v, g, beta, ends, scale, init=None):
    """out [tokens, v_heads, v_dim] and the final states [episodes, v_heads, v_dim, k_dim]."""
    q, k, v, g, beta = (np.asarray(x, np.float64) for x in (q, k, v, g, beta))
    group = v.shape[1] // k.shape[1]
    q, k = np.repeat(q, group, 1), np.repeat(k, group, 1)
    out = np.zeros(v.shape)
    final = np.zeros((len(ends), v.shape[1], v.shape[2], k.shape[2]))
    for e, (lo, hi) in enumerate(_spans(ends)):
        s = np.zeros(final.shape[1:]) if init is None else np.array(init[e], np.float64)
        for t in range(lo, hi):
            old = np.exp(g[t])[:, None, None] * s
            u = beta[t][:, None] * (v[t] - np.einsum("hvk,hk->hv", old, k[t]))
            s = old + u[:, :, None] * k[t][:, None, :]
            out[t] = scale * np.einsum("hvk,hk->hv", s, q[t])
        final[e] = s
    return out, final


def backward(q, k, v, g, beta, ends, scale, dout, init=None, d_final=None):
    """dq, dk, dv, dg, dbeta and the gradient of the initial states."""
    q, k, v, g, beta, dout = (np.asarray(x, np.float64) for x in (q, k, v, g, beta, dout))
    hk = k.shape[1]
    group = v.shape[1] // hk
    q, k = np.repeat(q, group, 1), np.repeat(k, group, 1)
    dq, dk, dv, dg, db = (np.zeros(x.shape) for x in (q, k, v, g, beta))
    d_init = np.zeros((len(ends), v.shape[1], v.shape[2], k.shape[2]))
    for e, (lo, hi) in enumerate(_spans(ends)):
        s = np.zeros(d_init.shape[1:]) if init is None else np.array(init[e], np.float64)
        before = []
        for t in range(lo, hi):
            before.append(s)
            old = np.exp(g[t])[:, None, None] * s
            u = beta[t][:, None] * (v[t] - np.einsum("hvk,hk->hv", old, k[t]))
            s = old + u[:, :, None] * k[t][:, None, :]
        ds = np.zeros(s.shape) if d_final is None else np.array(d_final[e], np.float64)
        for t in range(hi - 1, lo - 1, -1):
            old = np.exp(g[t])[:, None, None] * before.pop()
            err = v[t] - np.einsum("hvk,hk->hv", old, k[t])
            u = beta[t][:, None] * err
            new = old + u[:, :, None] * k[t][:, None, :]
            dq[t] = scale * np.einsum("hvk,hv->hk", new, dout[t])
            ds = ds + scale * dout[t][:, :, None] * q[t][:, None, :]
            du = np.einsum("hvk,hk->hv", ds, k[t])
            db[t] = (du * err).sum(-1)
            dv[t] = beta[t][:, None] * du
            dk[t] = np.einsum("hvk,hv->hk", ds, u) - np.einsum("hvk,hv->hk", old, dv[t])
            dold = ds - dv[t][:, :, None] * k[t][:, None, :]
            dg[t] = (dold * old).sum((-1, -2))
            ds = np.exp(g[t])[:, None, None] * dold
        d_init[e] = ds
    dq, dk = (x.reshape(x.shape[0], hk, group, x.shape[2]).sum(2) for x in (dq, dk))
    return dq, dk, dv, dg, db, d_init
