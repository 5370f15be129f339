"""How the selective scan cuts calls, on the host: every cut covers its call and fits the workspace."""
import ctypes as C
import random

import pytest

from _scan_cut import WHOLE, cut_of


@pytest.fixture(scope="module", autouse=True)
def lib():
    from offline_rl_step_gb300 import _abi, build
    build.build()
    return _abi.load()


def test_cuts_fit_their_workspace():
    rng = random.Random(0)
    log = lambda lo, hi: int(lo * (hi / lo) ** rng.random())  # noqa: E731
    whole = 0
    for _ in range(20000):
        groups = rng.choice((1, 1, 1, 2, 3, 8))
        channels = groups * 8 * log(1, 8192 // groups + 1)
        n = 4 * rng.randint(1, 16)
        episodes = log(1, 4000)
        if rng.random() < 0.5:      # lengths that divide the tokens into whole tiles
            tokens = episodes * 16 * log(1, 260)
        else:
            tokens = log(1, 3_000_000) - 1
        most = tokens + (0 if rng.random() < 0.5 else log(1, 100_000))
        sms, backward = rng.choice((1, 20, 132, 148, 152, 160)), rng.random() < 0.5
        c = cut_of((channels, n, groups), tokens, episodes, sms, backward, max_tokens=most)
        what = (channels, n, groups, tokens, episodes, sms, backward, c)
        assert c.used <= c.held, what
        assert c.seg % 16 == 0 and 64 <= c.seg <= 4096, what
        assert c.segments >= 1 and c.segments * c.seg >= tokens and (c.segments == 1 or (c.segments - 1) * c.seg < tokens), what
        per_block = 4 * (32 // c.lanes) * c.each
        assert 4 * c.lanes >= n and c.blocks == groups * -(-(channels // groups) // per_block), what
        whole += c.seg * episodes == tokens and c.segments > 1
    assert whole > 300      # the draw takes that path often enough


@pytest.mark.parametrize("case", list(WHOLE), ids=str)
def test_cases_of_whole_episodes(case):
    """What the GPU tests of this cut rely on, for the 152 SMs they run on."""
    shape, episodes, length, backward, each = WHOLE[case]
    c = cut_of(shape, episodes * length, episodes, 152, backward)
    assert c.seg == length and c.segments == episodes and c.each == each


def test_refusals(lib):
    from offline_rl_step_gb300 import _abi
    out = (C.c_int64 * 7)()
    ok = _abi.ScanShape(64, 16, 1, 0, 1)
    call = lib.ofrl_selftest_scan_cut
    assert call(C.byref(ok), 100, 1, 100, 152, 0, out) == _abi.OK
    assert call(None, 100, 1, 100, 152, 0, out) == _abi.EINVAL
    assert call(C.byref(_abi.ScanShape(60, 16, 1, 0, 1)), 100, 1, 100, 152, 0, out) == _abi.EUNSUPPORTED
    for bad in ((-1, 1, 100, 152, 0), (100, -1, 100, 152, 0), (100, 1, -1, 152, 0), (100, 1, 100, 0, 0), (100, 1, 100, 152, 2)):
        assert call(C.byref(ok), *bad, out) == _abi.EINVAL
    assert call(C.byref(ok), 100, 1, 100, 152, 0, None) == _abi.EINVAL
