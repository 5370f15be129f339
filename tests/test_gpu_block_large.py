"""State space blocks past 32-bit offsets: the last rows of calls of more than 2^31 elements are those of a call on
these rows alone."""
import pytest
import torch

from _gpu import need_gpu

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _room(gigabytes):
    need_gpu()
    if torch.cuda.mem_get_info()[0] < gigabytes * 2 ** 30:
        pytest.skip(f"needs {gigabytes} GB of free memory")


def test_convolution():
    import offline_rl_step_gb300 as ofrl
    _room(30)
    t, c, tail = 2 ** 21 + 300, 1040, 1000      # 2.18 billion elements
    gen = torch.Generator(device="cuda").manual_seed(0)
    x, dout = torch.zeros(t, c, device="cuda", dtype=BF), torch.zeros(t, c, device="cuda", dtype=BF)
    x[-tail:], dout[-tail:] = torch.randn(2, tail, c, device="cuda", generator=gen).to(BF)
    w = torch.randn(c, 4, device="cuda", generator=gen)
    ends = torch.tensor([t - tail // 2, t], dtype=torch.int32, device="cuda")
    short = torch.tensor([tail // 2, tail], dtype=torch.int32, device="cuda")
    ctx = ofrl.CausalConv(c, 4, "silu", "bf16", t, 2)
    out, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
    ofrl.conv_forward(ctx, x, w, ends, out)
    ofrl.conv_backward(ctx, x, w, ends, dout, dx, dw)
    o, g, wg = torch.empty(tail, c, device="cuda", dtype=BF), torch.empty(tail, c, device="cuda", dtype=BF), torch.empty_like(w)
    ofrl.conv_forward(ctx, x[-tail:], w, short, o)
    ofrl.conv_backward(ctx, x[-tail:], w, short, dout[-tail:], g, wg)
    assert torch.equal(out[-tail:], o) and torch.equal(dx[-tail:], g)
    # the same terms in another order, up to a thousand of them of either sign
    assert (dw - wg).norm() <= 1e-5 * wg.norm()
    assert (out[:t - tail] == 0).all()


def test_scan():
    import offline_rl_step_gb300 as ofrl
    _room(60)
    t, c, n, tail = 600_008, 512, 64, 2000      # 2.46 billion saved states
    gen = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(*s, device="cuda", generator=gen).to(BF)  # noqa: E731
    x, dt, z, dout, B, C = r(t, c), r(t, c), r(t, c), r(t, c), r(t, 1, n), r(t, 1, n)
    A = -torch.rand(c, n, device="cuda", generator=gen) - 0.5
    at = t - tail      # an episode of its own, so that nothing before counts
    ends = torch.tensor([at // 2, at, t], dtype=torch.int32, device="cuda")
    ctx = ofrl.SelectiveScan(c, n, 1, "bf16", True, t, 3)

    def both(rows, ends, states):
        a = [v[rows] for v in (x, dt)] + [A] + [v[rows] for v in (B, C)]
        out, gx, gd, gz = (torch.empty_like(a[0]) for _ in range(4))
        gB, gC, gA = torch.empty_like(a[3]), torch.empty_like(a[4]), torch.empty_like(A)
        final, saved = torch.empty(states, c, n, device="cuda"), ctx.saved(a[0].shape[0])
        ofrl.scan_forward(ctx, *a, ends, out, z=z[rows], final_state=final, saved=saved)
        ofrl.scan_backward(ctx, *a, ends, saved, dout[rows], gx, gd, gA, gB, gC, z=z[rows], dz=gz)
        return [out, gx, gd, gz, gB, gC], final

    whole, final = both(slice(None), ends, 3)
    part, last = both(slice(at, None), torch.tensor([tail], dtype=torch.int32, device="cuda"), 1)
    for a, b in zip(whole, part):
        # cut into segments of other lengths: decays multiply in another order, then a rounding to bf16
        assert (a[at:].float() - b.float()).norm() <= 2e-3 * b.float().norm()
    assert (final[2] - last[0]).norm() <= 1e-5 * last[0].norm()


def test_steps():
    import offline_rl_step_gb300 as ofrl
    _room(30)
    slots, c, n = 70_000, 512, 64      # 2.29 billion states
    state = torch.zeros(slots, c, n, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    x, dt, B, C, A = r(3, c), r(3, c), r(3, 1, n), r(3, 1, n), -torch.rand(c, n, device="cuda", generator=gen)
    idx = torch.tensor([slots - 1, 5, slots - 2], dtype=torch.int32, device="cuda")
    state[idx.long()] = r(3, c, n)
    ctx = ofrl.SelectiveScan(c, n, 1, "fp32", True, 0, 0, backward=False)
    small, out, want = state[idx.long()].clone(), torch.empty_like(x), torch.empty_like(x)
    ofrl.scan_step(ctx, x, dt, A, B, C, small, want)
    ofrl.scan_step(ctx, x, dt, A, B, C, state, out, slots=idx)
    assert torch.equal(out, want) and torch.equal(state[idx.long()], small)
    state[idx.long()] = 0
    assert not state.any()


def test_norms():
    import offline_rl_step_gb300 as ofrl
    _room(40)
    rows, c, tail = 2 ** 21 + 300, 1040, 500
    gen = torch.Generator(device="cuda").manual_seed(0)
    x, z, g = (torch.zeros(rows, c, device="cuda", dtype=BF) for _ in range(3))
    for v in (x, z, g):
        v[-tail:] = torch.randn(tail, c, device="cuda", generator=gen).to(BF)
    w, ctx = torch.rand(c, device="cuda", generator=gen) + 0.5, ofrl.BlockNorm(c, 1, "bf16")

    def run(op, back, *a):
        o = [torch.empty_like(a[0]) for _ in range(4)]
        dw = torch.empty_like(w)
        if op is ofrl.gated_norm:
            op(ctx, a[0], a[1], w, o[0])
            back(ctx, a[0], a[1], w, a[2], o[1], o[2], dw)
            return o[:3], dw
        op(ctx, a[0], a[1], w, o[0], o[1])
        back(ctx, a[0], a[1], w, a[2], o[2], o[3], dw)
        return o, dw

    for op, back in ((ofrl.gated_norm, ofrl.gated_norm_backward), (ofrl.residual_norm, ofrl.residual_norm_backward)):
        whole, dw = run(op, back, x, z, g)
        part, small = run(op, back, x[-tail:], z[-tail:], g[-tail:])
        assert all(torch.equal(a[-tail:], b) for a, b in zip(whole, part))
        assert (dw - small).norm() <= 1e-5 * small.norm()
        assert all((a[:rows - tail] == 0).all() for a in whole)
        del whole, part


def test_a_gradient_summed_over_long_segments():
    """dA of terms of one sign, over segments of up to 4096 tokens and 32768 in all.  With decays of about one half, a
    mean error of 5e-8 each makes the two factors of a term 1.0e-7 + 0.5e-7 and 1.0e-7 off.  Running sums of 128 terms
    round by 2.5e-8 of themselves a step, sqrt(128 / 3) times that in all: 1.6e-7; of the 32 sums of a segment and of
    the segments, 0.8e-7 and less.  The steps and A log2 e are rounded once, 3e-8 each, of no sign."""
    import numpy as np

    import offline_rl_step_gb300 as ofrl
    _room(20)
    t, c, n, few = 32768, 4864, 16, 64
    rng = np.random.default_rng(0)
    A = (-np.log(2) * rng.uniform(0.8, 1.2, (c, n))).astype(np.float32)
    gen = torch.Generator(device="cuda").manual_seed(0)
    dt = torch.rand(t, c, device="cuda", generator=gen) * 0.4 + 0.8
    x, b, a = torch.ones(t, c, device="cuda"), torch.ones(t, 1, n, device="cuda"), torch.from_numpy(A).cuda()
    ctx = ofrl.SelectiveScan(c, n, 1, "fp32", False, t, 1)
    saved, out, dx, ddt = ctx.saved(t), torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    da, db, dc = torch.empty_like(a), torch.empty_like(b), torch.empty_like(b)
    ends = torch.tensor([t], dtype=torch.int32, device="cuda")
    ofrl.scan_forward(ctx, x, dt, a, b, b, ends, out, saved=saved)
    ofrl.scan_backward(ctx, x, dt, a, b, b, ends, saved, x, dx, ddt, da, db, dc)
    got, steps, A = da[:few].double().cpu().numpy(), dt[:, :few].double().cpu().numpy(), A[:few].astype(np.float64)
    h, lam, want = np.zeros((few, n)), np.zeros((few, n)), np.zeros((few, n))
    past = np.empty((t, few, n))
    for i in range(t):
        past[i] = h
        h = np.exp(steps[i, :, None] * A) * h + steps[i, :, None]
    for i in range(t - 1, -1, -1):
        lam += 1
        decay = np.exp(steps[i, :, None] * A)
        want += steps[i, :, None] * lam * decay * past[i]
        lam *= decay
    assert np.linalg.norm(got - want) <= 6e-7 * np.linalg.norm(want)
