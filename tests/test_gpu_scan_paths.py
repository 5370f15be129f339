"""The selective scan where its paths differ: states that are joined while they grow, sums over long segments, steps, segments
that are whole episodes, rollouts of many tokens a CTA."""
import numpy as np
import pytest
import torch

from _block import ROUNDED, SCAN, check, dev, host, junk, scan_inputs
from _gpu import need_gpu
from _scan_cut import WHOLE, cut_of
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


@pytest.mark.parametrize("step", [0.001, 0.1])
def test_steps_summed_over_long_segments(step):
    """A segment of 4096 equal steps, whose sum S decays what comes before it by exp(A S) = 1 / e.  An addition rounds by
    at most 2^-24 of its result: a tile's 16 steps by sum(k / 16) = 8.5 of that, the 256 tiles of a segment by
    sum(k / 256) = 128.5, together 8.2e-6.  A S log2 e and the decay are rounded at 2^-23 and 2^-22, A and A log2 e at
    2^-24 each: 5e-7.  In one running sum the steps are 6e-5 off."""
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    if torch.cuda.mem_get_info()[0] < 12 * 2 ** 30:
        pytest.skip("needs 12 GB of free memory")
    t, c, n, seg = 3 * 4096, 6528, 64, 4096      # channels enough that a segment is as long as one may be
    gen = torch.Generator(device="cuda").manual_seed(0)
    dt = (step * 10 ** torch.rand(c, device="cuda", generator=gen)).expand(t, c).contiguous()
    A = (-1.0 / (dt[0] * seg)).view(c, 1).expand(c, n).contiguous()
    first, zero = torch.zeros(t, 1, n, device="cuda"), torch.zeros(t, c, device="cuda")
    first[:, :, 0] = 1
    ctx = ofrl.SelectiveScan(c, n, 1, "fp32", False, t, 2)
    out, saved, init = torch.empty_like(zero), ctx.saved(t), torch.ones(2, c, n, device="cuda")
    rate = A[:, 0].double() * dt[0].double()
    # forward, from the last token of the first segment over the second one
    ends = torch.tensor([seg - 1, t], dtype=torch.int32, device="cuda")
    ofrl.scan_forward(ctx, zero, dt, A, first, first, ends, out, init_state=init)
    assert (out[2 * seg] / torch.exp(rate * (seg + 2)) - 1).abs().max() <= 9e-6
    # gradients, from the first token of the third segment back
    ends = torch.tensor([2 * seg + 1, t], dtype=torch.int32, device="cuda")
    ofrl.scan_forward(ctx, zero, dt, A, first, first, ends, out, saved=saved)
    dx, ddt, dA, dB, dC = (torch.empty_like(v) for v in (zero, zero, A, first, first))
    ofrl.scan_backward(ctx, zero, dt, A, first, first, ends, saved, zero, dx, ddt, dA, dB, dC, d_final=init)
    assert (dx[seg - 1] / (dt[0] * torch.exp(rate * (seg + 1))) - 1).abs().max() <= 9e-6


@pytest.mark.parametrize("lo,hi", [(-80, -30), (-30, -10), (-10, -6), (-6, -4), (-4, -3), (-3, -2), (-2, -1), (-1, -0.5),
                                   (-0.5, -0.1), (-0.1, 0), (0, 0.1), (0.1, 0.5), (0.5, 1), (1, 3), (3, 10), (10, 30)], ids=str)
def test_mean_error_of_softplus(lo, hi):
    """Slow states sum their steps' mean error up, not each one's rounding.  The exponential's is at most 5.2e-8 over each
    of these ranges, 2.8e-8 of which is taken out; the polynomial is up to 5.4e-9 off.  The mean of 2^18 roundings, 7e-8
    each in the mean square, is 1.4e-10."""
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    t, c = 4096, 64
    v = np.random.default_rng(0).uniform(lo, hi, (t, c)).astype(np.float32)
    ctx = ofrl.SelectiveScan(c, 4, 1, "fp32", True, t, t, backward=False)
    one, first = torch.ones(t, c, device="cuda"), torch.zeros(t, 1, 4, device="cuda")
    first[:, :, 0] = 1
    # a token an episode, x = B = C = 1 in one state: the output is the step
    out, ends = junk(t, c), torch.arange(1, t + 1, dtype=torch.int32, device="cuda")
    ofrl.scan_forward(ctx, one, dev(v), -torch.ones(c, 4, device="cuda"), first, first, ends, out)
    v = v.astype(np.float64)
    want = np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))
    assert abs((host(out) / want - 1).mean()) <= 3e-8


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("case", list(WHOLE), ids=str)
def test_segments_of_whole_episodes(case, ragged):
    """Segments as long as the mean episode: episodes of that length, and as many of any length, hardly one of which ends
    where a segment does."""
    need_gpu()
    (c, n, groups), e, length, backward, each = WHOLE[case]
    t = e * length
    cut = cut_of((c, n, groups), t, e, torch.cuda.get_device_properties(0).multi_processor_count, backward)
    assert (cut.seg, cut.segments, cut.each) == (length, e, each)
    ln, dtype = [length] * e, "bf16"
    if ragged:
        at = np.sort(np.random.default_rng(e).integers(0, t + 1, e - 1))
        ln, dtype = [int(x) for x in np.diff(np.r_[0, at, t])], "fp32"
        assert max(ln) > 2 * length and min(ln) < length // 8
    d = scan_inputs(ln, c, n, groups, 12, dtype)
    _check(d, ln, dtype, _run(d, ln, dtype, slices=True))


def _one_token(d, state, softplus):
    """The step's outputs and states in 64 bits, a state a token."""
    x, dt, A, B, C, D, z, b = (d[k].astype(np.float64) for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias"))
    per = x.shape[1] // B.shape[1]
    delta = np.logaddexp(dt + b, 0.0) if softplus else dt + b
    h = np.exp(delta[:, :, None] * A) * state + (delta * x)[:, :, None] * np.repeat(B, per, 1)
    return ((h * np.repeat(C, per, 1)).sum(2) + D * x) * z / (1 + np.exp(-z)), h


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("c,n,groups", [(24, 4, 1), (24, 8, 3), (48, 16, 1), (144, 12, 2), (40, 32, 1), (264, 32, 1), (40, 44, 1),
                                        (16, 64, 2)])
def test_rollout_of_many_tokens(dtype, in_place, c, n, groups):
    """Four to six tokens a CTA, by a list of slots: a third of the tokens name none, in the middle of a CTA's tokens too.
    B and C of odd offset and stride in one of the two ways."""
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    lanes = cut_of((c, n, groups), 16, 1, sms, False).lanes
    columns = -(-c // (128 // lanes * min(lanes, 4)))
    ctas = -(-4 * sms // columns)      # along the tokens
    t = 5 * ctas + ctas // 2 + 1
    d = scan_inputs([t], c, n, groups, 21, dtype)
    r = np.random.default_rng(3)
    slots = t + 50
    at = r.permutation(slots)[:t].astype(np.int32)
    bad = r.random(t) < 1 / 3
    at[bad] = r.choice([-1, slots, -2 ** 31, 2 ** 31 - 1, slots + 7], bad.sum())
    before = np.float32(r.standard_normal((slots, c, n)))
    x, dt, B, C, z = (dev(d[k], dtype) for k in ("x", "dt", "B", "C", "z"))
    if in_place:
        wide = torch.zeros(t, 2 * groups * n + 3, device="cuda", dtype=B.dtype)
        wide[:, 1:] = torch.cat([B.flatten(1), C.flatten(1), B[:, 0, :2]], 1)
        B = wide[:, 1:1 + groups * n].unflatten(1, (groups, n))
        C = wide[:, 1 + groups * n:1 + 2 * groups * n].unflatten(1, (groups, n))
    out, state = junk(t, c, dtype=dtype), dev(before)
    new = state if in_place else torch.full_like(state, 7.0)
    ctx = ofrl.SelectiveScan(c, n, groups, dtype, True, 0, 0, backward=False)
    ofrl.scan_step(ctx, x, dt, dev(d["A"]), B, C, state, out, D=dev(d["D"]), z=z, dt_bias=dev(d["dt_bias"]),
                   new_state=None if in_place else new, slots=torch.from_numpy(at).cuda())
    assert ctx.poll_status()["bad_index"] == bad.sum()
    want, h = _one_token(d, before[np.where(bad, 0, at)], True)
    got, after = host(out), host(new)
    assert (got[bad] == 0).all()
    check(got[~bad], want[~bad], SCAN + ROUNDED[dtype], "out")
    check(after[at[~bad]], h[~bad], SCAN, "state")
    others = np.setdiff1d(np.arange(slots), at[~bad])
    assert (after[others] == (before[others] if in_place else 7.0)).all()
    if not in_place:
        assert np.array_equal(host(state), before.astype(np.float64))
