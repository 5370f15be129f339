"""Growth within a chunk of 64 tokens beyond what fp16 operands under common powers of two can hold, by positive log
decays or by keys with beta |k|^2 above two: outputs and states are those of the recurrence all the same, and gradients
either are right or not finite, never finite and wrong."""
import numpy as np
import pytest

from _delta import BOUND, STATE_BOUND, ends_of, inputs, off
from _gpu import need_gpu
from test_gpu_delta import GRAD_STATE_BOUND, LABELS, NAMES, ROUND, _run, _want

pytestmark = pytest.mark.gpu

LENGTHS = [64, 20, 0, 65]


def _bounds(dtype, strength):
    """Of outputs (eight tokens at a time), states and gradients.

    Decays: up to 2^16 of growth go through the chunk, whose first tokens' entries of P then have 18 bits with two planes
    (2e-5).  Keys: T's elements alternate in sign and their products with x cancel by 1 + 2 / (beta |k|^2 - 2), about
    twenty times for the smallest case here, through operands of 22 (11) bits: 1e-4 (1.5e-2).  Gradients may be far
    smaller than the products they are made of: ten times the usual bound."""
    out = (1e-4 if dtype == "fp32" else 1.5e-2) if strength else max(BOUND[dtype], 2e-5)
    return out, 1e-4 if strength else 2 * STATE_BOUND, 10 * BOUND[dtype]


def _inputs(dtype, hk, hv, dk, dv, g, strength, lengths=LENGTHS):
    d = inputs(lengths, hk, hv, dk, dv, seed=dk + dv, rnd=ROUND[dtype])
    r = np.random.default_rng(5)
    if g:
        d["g"] = ROUND[dtype](r.uniform(0.9 * g, 1.1 * g, d["g"].shape).astype(np.float32))
        d["q"] = d["k"].copy()
    if strength:      # keys near one direction: the state's part along it changes sign and grows
        k0 = r.standard_normal(dk)
        k = k0 / np.linalg.norm(k0) + 0.1 * r.standard_normal(d["k"].shape) / np.sqrt(dk)
        k *= np.sqrt(strength) / np.linalg.norm(k, axis=-1, keepdims=True)
        d["k"] = ROUND[dtype](k.astype(np.float32))
        d["q"] = d["k"].copy()
        d["beta"] = np.ones_like(d["beta"])
        d["g"] = np.zeros_like(d["g"])
    return d


def _sizes(d, lo, hi, e, scale):
    """Per token and head |dold| |old| and |du| |err|, of which dg and dbeta are the inner products (fp64)."""
    q, k, v, g, beta, dout = (np.float64(d[n][lo:hi]) for n in NAMES + ("dout",))
    group = v.shape[1] // k.shape[1]
    q, k = np.repeat(q, group, 1), np.repeat(k, group, 1)
    s, olds, errs = np.float64(d["init"][e]), [], []
    for t in range(hi - lo):
        olds.append(np.exp(g[t])[:, None, None] * s)
        errs.append(v[t] - np.einsum("hvk,hk->hv", olds[t], k[t]))
        s = olds[t] + (beta[t][:, None] * errs[t])[:, :, None] * k[t][:, None, :]
    ds, of_g, of_beta = np.float64(d["d_final"][e]), np.zeros(g.shape), np.zeros(g.shape)
    for t in range(hi - lo - 1, -1, -1):
        ds = ds + scale * dout[t][:, :, None] * q[t][:, None, :]
        du = np.einsum("hvk,hk->hv", ds, k[t])
        dold = ds - (beta[t][:, None] * du)[:, :, None] * k[t][:, None, :]
        of_beta[t] = np.linalg.norm(du, axis=1) * np.linalg.norm(errs[t], axis=1)
        of_g[t] = np.linalg.norm(dold, axis=(1, 2)) * np.linalg.norm(olds[t], axis=(1, 2))
        ds = np.exp(g[t])[:, None, None] * dold
    return of_g, of_beta


CASES = [(0.2, 0), (0.3, 0), (0.42, 0), (0.65, 0), (0, 2.3), (0, 2.56), (0, 3.0)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("hk,hv,dk,dv", [(1, 2, 64, 64), (1, 2, 128, 128), (1, 1, 40, 72)])
@pytest.mark.parametrize("g,strength", CASES)
def test_outputs_and_states(dtype, hk, hv, dk, dv, g, strength):
    need_gpu()
    d = _inputs(dtype, hk, hv, dk, dv, g, strength)
    bound, state_bound, _ = _bounds(dtype, strength)
    for states, grads in ((True, False), (False, False), (True, True), (False, True)):
        out, final = _run(d, LENGTHS, dtype, states=states, grads=grads)[:2]
        want = _want(d, LENGTHS, states=states)
        lo = 0
        for e, hi in enumerate(ends_of(LENGTHS)):
            for t in range(lo, hi, 8):      # early ones are far smaller than late ones
                x, y = out[t:min(t + 8, hi)], want[0][t:min(t + 8, hi)]
                assert off(x, y) <= bound, (e, t - lo, off(x, y))
            if states:
                assert off(final[e], want[1][e]) <= state_bound, (e, off(final[e], want[1][e]))
            lo = hi


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("hk,hv,dk,dv", [(1, 2, 64, 64), (1, 2, 128, 128), (1, 1, 40, 72)])
@pytest.mark.parametrize("g,strength", CASES)
def test_gradients_are_right_or_not_finite(dtype, hk, hv, dk, dv, g, strength):
    need_gpu()
    d = _inputs(dtype, hk, hv, dk, dv, g, strength)
    got, want = _run(d, LENGTHS, dtype), _want(d, LENGTHS)
    bound = _bounds(dtype, strength)[2]
    lo = 0
    for e, hi in enumerate(ends_of(LENGTHS)):
        sizes = dict(zip(("dg", "dbeta"), _sizes(d, lo, hi, e, 0.3)))
        for name, x, y in list(zip(LABELS, got, want))[2:]:
            for at in (slice(e, e + 1),) if name == "d_init" else [slice(c, min(c + 64, hi)) for c in range(lo, hi, 64)]:
                bad = ~np.isfinite(x[at])
                assert bad.all() or not bad.any(), f"{name} of episode {e}: {bad.mean():.2f} not finite"
                if g == 0.2:      # at most 2^20 in a chunk: inside what gradients of either type take
                    assert not bad.any(), name
                if not bad.any():
                    limit = max(bound, GRAD_STATE_BOUND * (name == "d_init" and dtype == "bf16")) * np.linalg.norm(y[at])
                    if name in sizes:      # of what the inner product is made of: 11 bits, or a few units of 22 and of fp32's sums
                        limit += (2.0 ** -11 if dtype == "bf16" else 2.0 ** -20) * np.linalg.norm(sizes[name][at.start - lo:at.stop - lo])
                    assert np.linalg.norm(x[at] - y[at]) <= limit, (name, e, off(x[at], y[at]))
        lo = hi


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (64, 128)])
def test_growth_within_one_part_of_a_long_episode(dtype, dk, dv):
    """Read in parts: growth of 2^40 within one of them, which the parts after it start from."""
    need_gpu()
    lengths = [1000]
    d = _inputs(dtype, 1, 1, dk, dv, 0, 0, lengths)
    d["g"][400:460] = ROUND[dtype](np.float32(0.46))
    d["g"][500:560] = ROUND[dtype](np.float32(-0.46))
    for states in (True, False):
        out, final = _run(d, lengths, dtype, states=states, grads=False)[:2]
        want = _want(d, lengths, states=states)
        for t in range(0, 1000, 8):
            assert off(out[t:t + 8], want[0][t:t + 8]) <= max(BOUND[dtype], 2e-5), (t, off(out[t:t + 8], want[0][t:t + 8]))
        if states:
            assert off(final, want[1]) <= 2 * STATE_BOUND
