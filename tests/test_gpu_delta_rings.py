"""Gradients of the gated delta rule where the chains' rings have one stage (more heads than SMs, at most 64 value
channels) and where a saving pass has two planes because a final state is asked for; fp32 tokens of very different size;
gradients against differences along themselves."""
import numpy as np
import pytest

from _delta import inputs
from _gpu import need_gpu
from test_gpu_delta import NAMES, ROUND, _compare, _run, _want

pytestmark = pytest.mark.gpu

MANY = [(i * 37) % 151 for i in range(45)]      # 0 to 150 tokens


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("states", [False, True])
@pytest.mark.parametrize("lengths,hk,hv,dk,dv", [(MANY, 4, 4, 64, 64), (MANY, 2, 4, 128, 64), (MANY, 1, 4, 24, 40),
                                                 ([1] * 300, 1, 2, 64, 64), ([1, 64] * 90, 1, 1, 128, 64),
                                                 ([65] * 80, 2, 4, 128, 128), ([2, 130] * 40, 1, 2, 40, 120)])
def test_learn_with_more_heads_than_sms(dtype, states, lengths, hk, hv, dk, dv):
    need_gpu()
    d = inputs(lengths, hk, hv, dk, dv, seed=dk + 2 * dv + len(lengths), rnd=ROUND[dtype])
    _compare(_run(d, lengths, dtype, states=states), _want(d, lengths, states=states), dtype)


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_fp32_tokens_of_very_different_size(dk, dv):
    """Within a chunk, keys, values and output gradients over four decades: two planes hold 22 bits of what is 2^-13 of
    its tile's largest (they end at 2^-39 of it)."""
    need_gpu()
    lengths = [150]
    d = inputs(lengths, 1, 1, dk, dv, seed=17)
    f = np.exp2(np.random.default_rng(0).integers(-13, 1, (150, 1, 1))).astype(np.float32)
    for name, x in (("k", f), ("v", f[::-1]), ("dout", np.roll(f, 7))):
        d[name] = d[name] * x
    _compare(_run(d, lengths, "fp32"), _want(d, lengths), "fp32")


@pytest.mark.parametrize("name", NAMES + ("init",))
def test_gradient_against_differences_along_itself(name):
    """Along the gradient the slope is |grad| |step|.  Central differences over h and h / 2 without their h^2 term leave
    h^4 (2^-24 for h = 1/64, times derivatives of the order of one); the outputs' error, 1e-5 of their norm and random
    over 1e4 of them, over h / 2 is 2e-5 of |out| |dout|, which the slopes of these inputs are at least a twentieth of."""
    need_gpu()
    lengths = [150, 20]
    d = inputs(lengths, 1, 2, 64, 64, seed=33)
    grad = dict(zip(NAMES + ("init",), _run(d, lengths, "fp32")[2:]))[name]
    step = grad * (np.linalg.norm(d[name]) / np.linalg.norm(grad))

    def slope(h):      # measured, and what the gradient says of the steps as fp32 made them
        f = []
        for sign in (1, -1):
            x = dict(d)
            x[name] = (d[name] + sign * h * step).astype(np.float32)
            o = _run(x, lengths, "fp32", grads=False)
            f.append(((o[0] * d["dout"]).sum() + (o[1] * d["d_final"]).sum(), x[name].astype(np.float64)))
        return (f[0][0] - f[1][0]) / (2 * h), ((f[0][1] - f[1][1]) * grad).sum() / (2 * h)

    (a, wa), (b, wb) = slope(2.0 ** -6), slope(2.0 ** -7)
    got, want = (4 * b - a) / 3, (4 * wb - wa) / 3
    assert abs(got - want) <= 2e-3 * abs(want), (name, got, want)
