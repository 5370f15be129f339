"""State space blocks in fp64 (numpy): short causal convolution, selective scan, gated norm, residual norm.

Episodes are packed: episode e's tokens lie between ends[e - 1] (0 for the first) and ends[e].
"""
import numpy as np


def _f64(*xs):
    return [None if x is None else np.asarray(x, np.float64) for x in xs]


def _spans(ends):
    start = 0
    for e in ends:
        yield start, int(e)
        start = int(e)


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def silu(x):
    return x * sigmoid(x)


def silu_slope(x):
    s = sigmoid(x)
    return s * (1.0 + x * (1.0 - s))


# ---- convolution: w [channels, width], the last tap takes the token itself ------------------------------------------


def conv_forward(x, w, bias, ends, act="silu", init=None):
    """out [tokens, channels], final states [episodes, channels, width - 1] and the sums before the activation."""
    x, w, bias, init = _f64(x, w, bias, init)
    t, d = x.shape
    k = w.shape[1]
    pre, final = np.zeros((t, d)), np.zeros((len(ends), d, k - 1))
    for e, (lo, hi) in enumerate(_spans(ends)):
        before = np.zeros((k - 1, d)) if init is None else init[e].T
        seen = np.concatenate([before, x[lo:hi]])
        for i in range(lo, hi):
            pre[i] = (seen[i - lo:i - lo + k] * w.T).sum(0) + (0.0 if bias is None else bias)
        final[e] = seen[len(seen) - (k - 1):].T
    return (silu(pre) if act == "silu" else pre), final, pre


def conv_backward(x, w, bias, ends, dout, act="silu", init=None, d_final=None):
    """dx, dw, dbias and the gradient of the initial states."""
    x, w, bias, dout, init, d_final = _f64(x, w, bias, dout, init, d_final)
    pre = conv_forward(x, w, bias, ends, act, init)[2]
    dpre = dout * silu_slope(pre) if act == "silu" else dout
    k, d = w.shape[1], x.shape[1]
    dx, dw, d_init, db = np.zeros(x.shape), np.zeros(w.shape), np.zeros((len(ends), d, k - 1)), np.zeros(d)
    for e, (lo, hi) in enumerate(_spans(ends)):
        before = np.zeros((k - 1, d)) if init is None else init[e].T
        seen = np.concatenate([before, x[lo:hi]])
        g = np.zeros(seen.shape)
        for i in range(hi - lo):
            g[i:i + k] += dpre[lo + i] * w.T
            dw += (dpre[lo + i] * seen[i:i + k]).T
            db += dpre[lo + i]
        if d_final is not None:
            g[len(g) - (k - 1):] += d_final[e].T
        d_init[e], dx[lo:hi] = g[:k - 1].T, g[k - 1:]
    return dx, dw, db, d_init


# ---- selective scan ---------------------------------------------------------------------------------------------------


def _deltas(dt, dt_bias, softplus):
    raw = dt + (0.0 if dt_bias is None else dt_bias)
    return (np.logaddexp(raw, 0.0) if softplus else raw), raw


def scan_forward(x, dt, A, B, C, ends, D=None, z=None, dt_bias=None, softplus=True, init=None):
    """out [tokens, channels] and final states [episodes, channels, state_dim]."""
    x, dt, A, B, C, D, z, dt_bias, init = _f64(x, dt, A, B, C, D, z, dt_bias, init)
    group = x.shape[1] // B.shape[1]
    delta, _ = _deltas(dt, dt_bias, softplus)
    y, final = np.zeros(x.shape), np.zeros((len(ends), *A.shape))
    for e, (lo, hi) in enumerate(_spans(ends)):
        h = np.zeros(A.shape) if init is None else init[e].copy()
        for t in range(lo, hi):
            h = np.exp(delta[t][:, None] * A) * h + (delta[t] * x[t])[:, None] * np.repeat(B[t], group, 0)
            y[t] = (h * np.repeat(C[t], group, 0)).sum(1)
        final[e] = h
    if D is not None:
        y = y + D * x
    return (y if z is None else y * silu(z)), final


def scan_backward(x, dt, A, B, C, ends, dout, D=None, z=None, dt_bias=None, softplus=True, init=None, d_final=None):
    """A dict of the gradients: x, dt, A, B, C, D, z, dt_bias, init."""
    x, dt, A, B, C, dout, D, z, dt_bias, init, d_final = _f64(x, dt, A, B, C, dout, D, z, dt_bias, init, d_final)
    groups = B.shape[1]
    group = x.shape[1] // groups
    delta, raw = _deltas(dt, dt_bias, softplus)
    gy = dout if z is None else dout * silu(z)
    y = np.zeros(x.shape)
    g = {"x": np.zeros(x.shape), "B": np.zeros(B.shape), "C": np.zeros(C.shape), "A": np.zeros(A.shape),
         "init": np.zeros((len(ends), *A.shape))}
    d_delta = np.zeros(x.shape)
    for e, (lo, hi) in enumerate(_spans(ends)):
        h = np.zeros(A.shape) if init is None else init[e].copy()
        kept = []
        for t in range(lo, hi):
            old = np.exp(delta[t][:, None] * A) * h
            h = old + (delta[t] * x[t])[:, None] * np.repeat(B[t], group, 0)
            y[t] = (h * np.repeat(C[t], group, 0)).sum(1)
            kept.append((old, h))
        adj = np.zeros(A.shape) if d_final is None else d_final[e].copy()
        for t in range(hi - 1, lo - 1, -1):
            old, h = kept.pop()
            b = np.repeat(B[t], group, 0)
            lam = adj + gy[t][:, None] * np.repeat(C[t], group, 0)
            g["C"][t] = (gy[t][:, None] * h).reshape(groups, group, -1).sum(1)
            g["B"][t] = (lam * (delta[t] * x[t])[:, None]).reshape(groups, group, -1).sum(1)
            to_input = (lam * b).sum(1)
            g["x"][t] = delta[t] * to_input
            d_delta[t] = x[t] * to_input + (lam * old * A).sum(1)
            g["A"] += lam * old * delta[t][:, None]
            adj = np.exp(delta[t][:, None] * A) * lam
        g["init"][e] = adj
    if D is not None:
        y = y + D * x
        g["x"] += D * gy
    g["D"] = (gy * x).sum(0)
    g["z"] = None if z is None else dout * y * silu_slope(z)
    g["dt"] = d_delta * sigmoid(raw) if softplus else d_delta
    g["dt_bias"] = g["dt"].sum(0)
    return g


# ---- norms --------------------------------------------------------------------------------------------------------------


def _grouped(x, groups):
    return x.reshape(x.shape[0], groups, -1)


def _norm(u, w, groups, eps):
    v = _grouped(u, groups)
    s = 1.0 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    return (v * s).reshape(u.shape) * w, s


def _norm_backward(u, w, groups, eps, e):
    """Gradients of w u / rms(u) with respect to u and w."""
    v = _grouped(u, groups)
    _, s = _norm(u, w, groups, eps)
    ew = _grouped(e * w, groups)
    du = s * (ew - v * s * s * (ew * v).mean(-1, keepdims=True))
    return du.reshape(u.shape), (e * (v * s).reshape(u.shape)).sum(0)


def gated_norm(x, z, w, groups=1, eps=1e-5, gate_first=False):
    x, z, w = _f64(x, z, w)
    if gate_first:
        return _norm(x * silu(z), w, groups, eps)[0]
    return _norm(x, w, groups, eps)[0] * silu(z)


def gated_norm_backward(x, z, w, dout, groups=1, eps=1e-5, gate_first=False):
    """dx, dz, dw."""
    x, z, w, dout = _f64(x, z, w, dout)
    gate = silu(z)
    if gate_first:
        du, dw = _norm_backward(x * gate, w, groups, eps, dout)
        return du * gate, du * x * silu_slope(z), dw
    dx, dw = _norm_backward(x, w, groups, eps, dout * gate)
    return dx, dout * _norm(x, w, groups, eps)[0] * silu_slope(z), dw


def residual_norm(x, residual, w, scale=None, groups=1, eps=1e-5):
    """The sum and its norm."""
    x, residual, w, scale = _f64(x, residual, w, scale)
    h = residual + (x if scale is None else scale * x)
    return h, _norm(h, w, groups, eps)[0]


def residual_norm_backward(x, residual, w, dout, scale=None, d_sum=None, groups=1, eps=1e-5):
    """dx, dresidual, dw, dscale."""
    x, residual, w, dout, scale, d_sum = _f64(x, residual, w, dout, scale, d_sum)
    h, _ = residual_norm(x, residual, w, scale, groups, eps)
    dh, dw = _norm_backward(h, w, groups, eps, dout)
    if d_sum is not None:
        dh = dh + d_sum
    return (dh if scale is None else scale * dh), dh, dw, (None if scale is None else (dh * x).sum(0))
