"""The gated delta rule with positive log decays: states that grow, within a chunk, over chunks and after a reset.

Bounds are those of decaying states: a chunk's decays are differences of exact sums, every operand is scaled by its
tile's largest element, and growth by 2^9 to 2^16 within a chunk of 64 tokens leaves what is smallest in it, an output of
the chunk's first tokens, within the 22 (11) bits that the largest one has (elements down to 2^-17 of their tile's largest
keep 21 of them, 2^-27 keeps 11).  Episodes are compared one by one: a long one outgrows a short one by e^13."""
import numpy as np
import pytest

from _delta import BOUND, ends_of, inputs
from _gpu import need_gpu
from test_gpu_delta import NAMES, ROUND, _compare, _run, _want

pytestmark = pytest.mark.gpu

LENGTHS = [130, 5, 0, 64, 65]


def _growing(lengths, hk, hv, dk, dv, dtype, low, high, along=False, seed=0):
    d = inputs(lengths, hk, hv, dk, dv, seed=seed + dk + dv, rnd=ROUND[dtype])
    r = np.random.default_rng(seed)
    d["g"] = ROUND[dtype](r.uniform(low, high, d["g"].shape).astype(np.float32))
    if along:      # queries along the keys of their token: the largest products
        d["q"] = d["k"].copy()
    return d


def _dg_terms(d, lo, hi, e, scale, states):
    """Per token and head |dold| |old|, of which dg = <dold, old> is the inner product (fp64)."""
    q, k, v, g, beta, dout = (np.float64(d[n][lo:hi]) for n in NAMES + ("dout",))
    group = v.shape[1] // k.shape[1]
    q, k = np.repeat(q, group, 1), np.repeat(k, group, 1)
    s = np.float64(d["init"][e]) * states
    olds = []
    for t in range(hi - lo):
        olds.append(np.exp(g[t])[:, None, None] * s)
        u = beta[t][:, None] * (v[t] - np.einsum("hvk,hk->hv", olds[t], k[t]))
        s = olds[t] + u[:, :, None] * k[t][:, None, :]
    ds, size = np.float64(d["d_final"][e]) * states, np.zeros(g.shape)
    for t in range(hi - lo - 1, -1, -1):
        ds = ds + scale * dout[t][:, :, None] * q[t][:, None, :]
        dold = ds - (beta[t][:, None] * np.einsum("hvk,hk->hv", ds, k[t]))[:, :, None] * k[t][:, None, :]
        size[t] = np.linalg.norm(dold, axis=(1, 2)) * np.linalg.norm(olds[t], axis=(1, 2))
        ds = np.exp(g[t])[:, None, None] * dold
    return size


def _check(d, lengths, dtype, **kw):
    states = kw.get("states", True)
    got, want = _run(d, lengths, dtype, **kw), _want(d, lengths, states=states)
    lo = 0
    for e, hi in enumerate(ends_of(lengths)):
        part = lambda x, tokens: None if x is None else x[lo:hi] if tokens else x[e:e + 1]
        tokens = (True, False, True, True, True, True, True, False)
        g, w = ([part(x, t) for x, t in zip(y, tokens)] for y in (got, want))
        if dtype == "bf16" and len(g) > 2 and hi > lo:
            # An inner product of two matrices that grow, one forward and one back, may be far smaller than they are;
            # operands of 11 bits leave it off by 2^-11 of their sizes beside what its own rounding does.
            slack = 2.0 ** -11 * np.linalg.norm(_dg_terms(d, lo, hi, e, 0.3, states))
            off = np.linalg.norm(g[5] - w[5])
            assert np.isfinite(g[5]).all() and off <= BOUND[dtype] * np.linalg.norm(w[5]) + slack, f"dg {e}: {off:.3g}"
            g[5] = None
        _compare(g, w, dtype)
        lo = hi


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("hk,hv,dk,dv", [(1, 2, 64, 64), (2, 4, 128, 128), (1, 1, 40, 72), (1, 2, 64, 16)])
@pytest.mark.parametrize("low,high", [(0.08, 0.14), (-0.3, 0.3)])
@pytest.mark.parametrize("grads", [True, False])
def test_growth(dtype, hk, hv, dk, dv, low, high, grads):
    need_gpu()
    d = _growing(LENGTHS, hk, hv, dk, dv, dtype, low, high, along=True)
    for states in (True, False):
        _check(d, LENGTHS, dtype, states=states, grads=grads)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("dv", [64, 128])
def test_growth_by_2_16_within_a_chunk(dtype, dv):
    """0.17 a token, 2^16 over 64 tokens."""
    need_gpu()
    d = _growing([64, 60], 1, 2, 64, dv, dtype, 0.16, 0.18, along=True, seed=1)
    for grads in (True, False):
        _check(d, [64, 60], dtype, grads=grads)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("dv", [64, 128])
def test_growth_after_a_reset(dtype, dv):
    need_gpu()
    lengths = [100, 150]
    d = _growing(lengths, 1, 2, 64, dv, dtype, 0.05, 0.15, along=True, seed=2)
    for t in (0, 40, 64, 100, 199):
        d["g"][t, t % 2] = -np.inf
    for grads in (True, False):
        _check(d, lengths, dtype, grads=grads)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_growth_over_a_long_episode(dtype, dk, dv):
    """Read in parts; growth and decay in turn, by e^6 each."""
    need_gpu()
    lengths = [1000]
    d = _growing(lengths, 1, 1, dk, dv, dtype, 0.08, 0.12, along=True, seed=3)
    sign = np.where(np.arange(1000) // 60 % 2 == 0, 1.0, -1.0).astype(np.float32)[:, None]
    d["g"] = d["g"] * sign
    for states in (True, False):
        _check(d, lengths, dtype, states=states, grads=False)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_reading_and_stepping_agree(dtype):
    """What the chunks give is what one token after the other gives."""
    import torch
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    n = 70
    d = _growing([n], 1, 2, 64, 64, dtype, 0.08, 0.1, along=True, seed=4)
    want = _want(d, [n], states=False)
    out = _run(d, [n], dtype, states=False, grads=True)[0]
    dt = {"fp32": torch.float32, "bf16": torch.bfloat16}[dtype]
    x = [torch.from_numpy(np.ascontiguousarray(d[name])).cuda().to(dt) for name in NAMES]
    ctx = ofrl.DeltaRule(1, 2, 64, 64, dtype, max_tokens=0, max_episodes=0, backward=False)
    state, one = torch.zeros(1, 2, 64, 64, device="cuda"), torch.empty(1, 2, 64, device="cuda", dtype=dt)
    stepped = []
    for t in range(n):
        ofrl.delta_step(ctx, *[y[t:t + 1] for y in x], state, one, scale=0.3)
        stepped.append(one.double().cpu().numpy()[0])
    ctx.close()
    for got in (out, np.stack(stepped)):
        _compare([got], want[:1], dtype)
