"""Non-finite tokens in the gated delta rule: what the recurrence leaves finite has to be right, and the rest not finite.

The recurrence in 64 bits says which outputs, states and gradients a NaN or an infinity reaches: in the value channel of
an element of v, or in all channels of a token's k, g or beta, everything from that token on, and of q that token alone.
Tokens before it, in its own chunk too, other channels and other episodes see nothing of it."""
import numpy as np
import pytest

from _delta import BOUND, STATE_BOUND, ends_of, inputs
from _gpu import need_gpu
from oracle import delta
from test_gpu_delta import GRAD_STATE_BOUND, LABELS, NAMES, ROUND, _run, _want

pytestmark = pytest.mark.gpu

LENGTHS = [20, 150, 0, 70]
SHAPES = [(1, 2, 64, 64), (2, 4, 128, 128), (1, 1, 40, 72), (1, 1, 128, 24)]


def _same_where_finite(got, want, bound, what):
    finite = np.isfinite(want)
    bad = np.isfinite(got) != finite
    assert not bad.any(), f"{what}: {np.count_nonzero(bad & finite)} spoilt, {np.count_nonzero(bad & ~finite)} not marked"
    g, w = np.where(finite, got, 0.0), np.where(finite, want, 0.0)
    n = np.linalg.norm(w)
    assert np.linalg.norm(g - w) <= bound * n, f"{what}: off by {np.linalg.norm(g - w) / n:.3g}"


def _compare(got, want, dtype):
    for name, x, y in zip(LABELS, got, want):
        if x is not None:
            _same_where_finite(x, y, STATE_BOUND if name == "final" or (name == "d_init" and dtype == "fp32") else
                               GRAD_STATE_BOUND if name == "d_init" else BOUND[dtype], name)


def _put(d, kind, t):
    value = {"nan": np.nan, "inf": np.inf, "-inf": -np.inf}[kind.split()[1]]
    name = kind.split()[0]
    if name in ("g", "beta"):
        d[name][t, 0] = value
    else:
        d[name][t, 0, 5] = value


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("hk,hv,dk,dv", SHAPES)
@pytest.mark.parametrize("kind", ["v nan", "v -inf", "k nan", "k inf", "q nan", "g nan", "g inf", "beta nan", "beta inf"])
def test_tokens_before_see_nothing_of_it(dtype, hk, hv, dk, dv, kind):
    need_gpu()
    for t in (20 + 70, 20 + 63, 20, 170):      # inside a chunk, its last token, an episode's first tokens
        d = inputs(LENGTHS, hk, hv, dk, dv, seed=dk + dv, rnd=ROUND[dtype])
        _put(d, kind, t)
        a = [d[n] for n in NAMES]
        with np.errstate(all="ignore"):
            want = [list(delta.forward(*a, ends_of(LENGTHS), 0.3, init=d["init"])),
                    list(delta.forward(*a, ends_of(LENGTHS), 0.3))]
        _compare(_run(d, LENGTHS, dtype, grads=False), want[0], dtype)
        _compare(_run(d, LENGTHS, dtype, states=False, grads=False), want[1][:1] + [None], dtype)
        _compare(_run(d, LENGTHS, dtype)[:2], want[0], dtype)
        _compare(_run(d, LENGTHS, dtype, states=False)[:2], want[1][:1] + [None], dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("hk,hv,dk,dv", SHAPES)
@pytest.mark.parametrize("kind", ["v nan", "v inf"])
def test_gradients_of_tokens_before_see_nothing_of_it(dtype, hk, hv, dk, dv, kind):
    need_gpu()
    for t in (20 + 70, 20 + 63, 20, 170):
        d = inputs(LENGTHS, hk, hv, dk, dv, seed=dk + dv + 1, rnd=ROUND[dtype])
        _put(d, kind, t)
        with np.errstate(all="ignore"):
            want = _want(d, LENGTHS)
        _compare(_run(d, LENGTHS, dtype), want, dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("hk,hv,dk,dv", [(1, 1, 64, 64), (1, 1, 128, 128)])
def test_long_episodes_and_states_that_are_not_finite(dtype, hk, hv, dk, dv):
    """Read in parts: a bad value in one part reaches the later ones; an infinite element of an initial state its row."""
    need_gpu()
    lengths = [1000]
    for kind, t in (("v inf", 500), ("k nan", 333), ("g inf", 901), (None, None)):
        d = inputs(lengths, hk, hv, dk, dv, seed=dk + dv + 2, rnd=ROUND[dtype])
        d["init"][0, 0, 3, 7] = np.inf
        if kind:
            d["init"][0, 0, 3, 7] = 0.0
            _put(d, kind, t)
        with np.errstate(all="ignore"):
            want = list(delta.forward(*[d[n] for n in NAMES], ends_of(lengths), 0.3, init=d["init"]))
        _compare(_run(d, lengths, dtype, grads=False), want, dtype)
