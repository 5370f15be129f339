"""Queries far larger and far smaller than one: only their outputs and the gradients of what they read scale with them."""
import numpy as np
import pytest

from _delta import inputs
from _gpu import need_gpu
from test_gpu_delta import ROUND, _compare, _run, _want

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
@pytest.mark.parametrize("size", [2.0 ** 100, 2.0 ** -100])
def test_queries_of_any_size(dtype, dk, dv, size):
    need_gpu()
    lengths = [130, 40]
    d = inputs(lengths, 1, 2, dk, dv, seed=41, rnd=ROUND[dtype])
    d["q"] = (d["q"] * np.float32(size)).astype(np.float32)      # powers of two: exact
    d["dout"] = (d["dout"] / np.float32(size)).astype(np.float32)
    _compare(_run(d, lengths, dtype), _want(d, lengths), dtype)
    _compare(_run(d, lengths, dtype, grads=False), _want(d, lengths), dtype)
