"""The fp64 oracle of state space blocks against torch's autograd, written apart from it, and against differences."""
import numpy as np
import pytest
import torch
import torch.nn.functional as F

from oracle import block

R = np.random.default_rng(5)


def _t(x):
    return torch.tensor(np.asarray(x), dtype=torch.float64, requires_grad=True)


def _close(got, want):
    np.testing.assert_allclose(got, want.detach().numpy() if isinstance(want, torch.Tensor) else want, rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("act", ["silu", "none"])
def test_conv_against_torch(width, act):
    """torch's convolution over each episode by itself, with its initial inputs in front."""
    lengths, d = [5, 0, 1, 2, 9], 6
    t, ends = sum(lengths), np.cumsum(lengths)
    x, w, b = _t(R.standard_normal((t, d))), _t(R.standard_normal((d, width))), _t(R.standard_normal(d))
    init = _t(R.standard_normal((len(lengths), d, width - 1)))
    dout, d_final = R.standard_normal((t, d)), R.standard_normal((len(lengths), d, width - 1))
    outs, finals, lo = [], [], 0
    for e, n in enumerate(lengths):
        seen = torch.cat([init[e], x[lo:lo + n].T], 1)
        if n:
            outs.append(F.conv1d(seen[None], w[:, None], b, groups=d)[0].T)
        finals.append(seen[:, seen.shape[1] - (width - 1):])
        lo += n
    out, final = torch.cat(outs), torch.stack(finals)
    out = F.silu(out) if act == "silu" else out
    ((out * torch.tensor(dout)).sum() + (final * torch.tensor(d_final)).sum()).backward()
    args = [v.detach().numpy() for v in (x, w, b)]
    got, got_final, _ = block.conv_forward(*args, ends, act, init.detach().numpy())
    _close(got, out)
    _close(got_final, final)
    for g, v in zip(block.conv_backward(*args, ends, dout, act, init.detach().numpy(), d_final), (x, w, b, init)):
        _close(g, v.grad)


def _scan_torch(x, dt, A, B, C, lengths, D, z, dt_bias, softplus, init):
    """The scan as one matrix product per episode: h_t is a sum over the tokens before it."""
    t, d = x.shape
    group = d // B.shape[1]
    raw = dt if dt_bias is None else dt + dt_bias
    delta = F.softplus(raw) if softplus else raw
    ys, finals, lo = [], [], 0
    for e, n in enumerate(lengths):
        s = slice(lo, lo + n)
        cum = torch.cat([torch.zeros(1, d, dtype=torch.float64), delta[s].cumsum(0)])
        h = []
        for i in range(n + 1):
            v = torch.exp(cum[i][:, None] * A) * (init[e] if init is not None else 0.0 * A)
            for j in range(i):
                v = v + torch.exp((cum[i] - cum[j + 1])[:, None] * A) * (delta[lo + j] * x[lo + j])[:, None] * \
                    B[lo + j].repeat_interleave(group, 0)
            h.append(v)
        ys += [(h[i + 1] * C[lo + i].repeat_interleave(group, 0)).sum(1) for i in range(n)]
        finals.append(h[n])
        lo += n
    y = torch.stack(ys)
    if D is not None:
        y = y + D * x
    return (y if z is None else y * F.silu(z)), torch.stack(finals)


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("parts", [("D", "z", "dt_bias", "init"), ("z",), ()])
def test_scan_against_torch(softplus, parts):
    lengths, d, n, groups = [4, 0, 1, 6], 6, 3, 2
    t, ends = sum(lengths), np.cumsum(lengths)
    v = {"x": _t(R.standard_normal((t, d))), "dt": _t(R.standard_normal((t, d)) * 0.5 + (0.0 if softplus else 0.5)),
         "A": _t(-R.uniform(0.2, 2.0, (d, n))), "B": _t(R.standard_normal((t, groups, n))),
         "C": _t(R.standard_normal((t, groups, n))), "D": _t(R.standard_normal(d)), "z": _t(R.standard_normal((t, d))),
         "dt_bias": _t(R.standard_normal(d)), "init": _t(R.standard_normal((len(lengths), d, n)))}
    more = {k: (v[k] if k in parts else None) for k in ("D", "z", "dt_bias", "init")}
    core = [v[k] for k in ("x", "dt", "A", "B", "C")]
    out, final = _scan_torch(*core, lengths, softplus=softplus, **more)
    dout, d_final = R.standard_normal((t, d)), R.standard_normal((len(lengths), d, n))
    ((out * torch.tensor(dout)).sum() + (final * torch.tensor(d_final)).sum()).backward()
    host = [x.detach().numpy() for x in core]
    more = {k: None if x is None else x.detach().numpy() for k, x in more.items()}
    got, got_final = block.scan_forward(*host, ends, softplus=softplus, **more)
    _close(got, out)
    _close(got_final, final)
    g = block.scan_backward(*host, ends, dout, softplus=softplus, d_final=d_final, **more)
    for k in ("x", "dt", "A", "B", "C") + tuple(parts):
        _close(g[k], v[k].grad)


def test_scan_closed_form():
    """One channel, one state, constant input: a geometric sum."""
    t, a, b = 30, -0.7, 0.4
    delta = 0.25
    r = np.exp(delta * a)
    one = np.ones((t, 1))
    out, final = block.scan_forward(one, delta * one, [[a]], b * one[:, :, None], one[:, :, None], [t], softplus=False)
    want = delta * b * (1 - r ** np.arange(1, t + 1)) / (1 - r)
    np.testing.assert_allclose(out[:, 0], want, rtol=1e-13)
    np.testing.assert_allclose(final[0, 0, 0], want[-1], rtol=1e-13)


@pytest.mark.parametrize("groups", [1, 3])
@pytest.mark.parametrize("gate_first", [False, True])
def test_gated_norm_against_torch(groups, gate_first):
    x, z, w = _t(R.standard_normal((7, 12))), _t(R.standard_normal((7, 12))), _t(R.standard_normal(12))
    dout = R.standard_normal((7, 12))
    u = x * F.silu(z) if gate_first else x
    out = F.rms_norm(u.view(7, groups, -1), (12 // groups,), eps=1e-3).reshape(7, 12) * w
    out = out if gate_first else out * F.silu(z)
    (out * torch.tensor(dout)).sum().backward()
    host = [v.detach().numpy() for v in (x, z, w)]
    _close(block.gated_norm(*host, groups, 1e-3, gate_first), out)
    for g, v in zip(block.gated_norm_backward(*host, dout, groups, 1e-3, gate_first), (x, z, w)):
        _close(g, v.grad)


@pytest.mark.parametrize("scaled", [False, True])
def test_residual_norm_against_torch(scaled):
    x, r, w, s = (_t(R.standard_normal(k)) for k in ((5, 8), (5, 8), 8, 8))
    dout, dh = R.standard_normal((5, 8)), R.standard_normal((5, 8))
    h = r + (s * x if scaled else x)
    out = F.rms_norm(h, (8,), eps=1e-3) * w
    ((out * torch.tensor(dout)).sum() + (h * torch.tensor(dh)).sum()).backward()
    host = [v.detach().numpy() for v in (x, r, w)]
    scale = s.detach().numpy() if scaled else None
    got_h, got = block.residual_norm(*host, scale, eps=1e-3)
    _close(got_h, h)
    _close(got, out)
    g = block.residual_norm_backward(*host, dout, scale, dh, eps=1e-3)
    for a, v in zip(g, (x, r, w) + ((s,) if scaled else ())):
        _close(a, v.grad)


def test_scan_gradients_against_differences():
    lengths, d, n = [3, 4], 2, 2
    t, ends = 7, np.cumsum(lengths)
    v = {"x": R.standard_normal((t, d)), "dt": R.standard_normal((t, d)), "A": -R.uniform(0.2, 2.0, (d, n)),
         "B": R.standard_normal((t, 1, n)), "C": R.standard_normal((t, 1, n)), "D": R.standard_normal(d),
         "z": R.standard_normal((t, d)), "dt_bias": R.standard_normal(d), "init": R.standard_normal((2, d, n))}
    dout, d_final = R.standard_normal((t, d)), R.standard_normal((2, d, n))

    def loss(u):
        out, final = block.scan_forward(*[u[k] for k in ("x", "dt", "A", "B", "C")], ends, u["D"], u["z"], u["dt_bias"],
                                        True, u["init"])
        return (out * dout).sum() + (final * d_final).sum()

    g = block.scan_backward(*[v[k] for k in ("x", "dt", "A", "B", "C")], ends, dout, v["D"], v["z"], v["dt_bias"], True,
                            v["init"], d_final)
    for k in v:
        step = R.standard_normal(v[k].shape)
        eps = 1e-6
        up, down = dict(v), dict(v)
        up[k], down[k] = v[k] + eps * step, v[k] - eps * step
        np.testing.assert_allclose((loss(up) - loss(down)) / (2 * eps), (g[k] * step).sum(), rtol=1e-6, atol=1e-7)
