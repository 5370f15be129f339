"""The gated delta rule over many episodes: what few of them never reach (one CTA per head for wide values, token by
token or chunked by estimate, parts of an episode whose chunks do not divide evenly)."""
import pytest

from _delta import inputs
from _gpu import need_gpu
from test_gpu_delta import ROUND, _compare, _run, _want

pytestmark = pytest.mark.gpu

MANY = [(i * 37) % 151 for i in range(45)]      # 0 to 150 tokens


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("states", [False, True])
@pytest.mark.parametrize("hk,hv,dk,dv", [(2, 4, 128, 128), (1, 4, 64, 120), (2, 6, 40, 72), (4, 4, 16, 64)])
def test_many_episodes_read(dtype, states, hk, hv, dk, dv):
    need_gpu()
    d = inputs(MANY, hk, hv, dk, dv, seed=dk + dv, rnd=ROUND[dtype])
    _compare(_run(d, MANY, dtype, states=states, grads=False), _want(d, MANY, states=states), dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("hk,hv,dk,dv", [(2, 4, 128, 128), (1, 4, 64, 72)])
def test_many_episodes_learn(dtype, hk, hv, dk, dv):
    need_gpu()
    d = inputs(MANY, hk, hv, dk, dv, seed=dk + dv + 1, rnd=ROUND[dtype])
    _compare(_run(d, MANY, dtype), _want(d, MANY), dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("lengths", [[1] * 300, [3] * 200 + [0], [0] * 50 + [17] * 50 + [200], [33, 2] * 40])
@pytest.mark.parametrize("hk,hv,dk,dv", [(1, 2, 128, 72), (1, 1, 24, 16), (2, 2, 64, 64)])
def test_short_episodes_read(dtype, lengths, hk, hv, dk, dv):
    need_gpu()
    d = inputs(lengths, hk, hv, dk, dv, seed=len(lengths), rnd=ROUND[dtype])
    for states in (False, True):
        _compare(_run(d, lengths, dtype, states=states, grads=False), _want(d, lengths, states=states), dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("lengths", [[768], [64 * 13 + 1], [1000, 1000, 1001]])
def test_parts_that_do_not_divide_evenly(dtype, lengths):
    need_gpu()
    d = inputs(lengths, 1, 2, 64, 64, seed=len(lengths), rnd=ROUND[dtype])
    for states in (False, True):
        _compare(_run(d, lengths, dtype, states=states, grads=False), _want(d, lengths, states=states), dtype)
