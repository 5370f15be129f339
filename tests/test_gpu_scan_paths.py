"""The selective scan where its paths differ: states that are joined while they grow, sums over long segments, rollouts
of many tokens a CTA, segments that are whole episodes."""
import numpy as np
import pytest
import torch

from _block import scan_inputs
from _gpu import need_gpu
from test_gpu_scan import _check, _run

pytestmark = pytest.mark.gpu


def test_a_state_of_zero_stays_where_others_would_grow():
    """A above zero: a segment's decay passes what fp32 holds, the state that it meets is zero.  Forward nothing comes in
    before the last five tokens, backward nothing behind the first five; what does grows by exp(5) a token at most."""
    need_gpu()
    ln = [2000, 90]
    d = scan_inputs(ln, 16, 16, 1, 4, "fp32", softplus=False)
    d["A"] = np.abs(d["A"]) / 5                       # 0.1 to 2
    d["dt"][:2000] = 2.0 + 0.5 * np.float32(np.random.default_rng(1).random((2000, 16)))
    d["dt"][2000:] = 0.01
    d["x"][:1995] = 0
    d["dout"][5:2000] = 0
    parts = ("D", "z")
    got = _run(d, ln, "fp32", parts, states=False, softplus=False)
    assert all(np.isfinite(v).all() for v in got.values() if v is not None)
    _check(d, ln, "fp32", got, parts, states=False, softplus=False)
