"""Offsets past 2^31 elements: the last episodes of a very long call give what they give by themselves."""
import pytest
import torch

from _delta import BOUND, check
from _gpu import need_gpu

pytestmark = pytest.mark.gpu


def _tokens(n, hk, hv, dim, gen):
    new = lambda *s: torch.randn(*s, device="cuda", generator=gen, dtype=torch.bfloat16)  # noqa: E731
    q, k = new(n, hk, dim) * dim ** -0.5, new(n, hk, dim) * dim ** -0.5
    return [q, k, new(n, hv, dim), -0.1 * new(n, hv).abs(), new(n, hv).sigmoid()]


def test_forward_and_backward():
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    hk, hv, dim, length, n_ep = 2, 20, 128, 256, 3290
    n = n_ep * length
    assert n * hv * dim > 2 ** 31
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GB of free device memory")
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = _tokens(n, hk, hv, dim, gen)
    dout = torch.randn(n, hv, dim, device="cuda", generator=gen, dtype=torch.bfloat16)

    def run(x, dout, episodes):
        ends = torch.arange(1, episodes + 1, device="cuda", dtype=torch.int32) * length
        ctx = ofrl.DeltaRule(hk, hv, dim, dim, "bf16", max_tokens=episodes * length, max_episodes=episodes)
        out, saved = torch.empty_like(dout), ctx.saved(episodes * length, episodes)
        grads = [torch.empty_like(t) for t in x]
        ofrl.delta_forward(ctx, *x, ends, out, saved=saved)
        ofrl.delta_backward(ctx, *x, ends, saved, dout, *grads)
        assert ctx.poll_status() == {"bad_index": 0, "timeout": 0}
        ctx.close()
        return [t[-2 * length:].double().cpu().numpy() for t in (out, *grads)]

    got = run(x, dout, n_ep)
    want = run([t[-2 * length:].contiguous() for t in x], dout[-2 * length:].contiguous(), 2)
    for name, a, b in zip(("out", "dq", "dk", "dv", "dg", "dbeta"), got, want):
        check(a, b, 2 * BOUND["bf16"], name)      # each side within its bound of the recurrence


def test_step_slots():
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    heads, dim, slots = 20, 128, 6600
    assert slots * heads * dim * dim > 2 ** 31
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB of free device memory")
    gen = torch.Generator(device="cuda").manual_seed(3)
    ctx = ofrl.DeltaRule(heads, heads, dim, dim, "bf16", max_tokens=0, max_episodes=0, backward=False)
    x = _tokens(3, heads, heads, dim, gen)
    state = torch.zeros(slots, heads, dim, dim, device="cuda")
    at = [0, slots - 1, slots // 2]
    for i in at:
        state[i] = torch.randn(heads, dim, dim, device="cuda", generator=gen)
    small, out, out_small = state[at].clone(), torch.empty_like(x[2]), torch.empty_like(x[2])
    ofrl.delta_step(ctx, *x, state, out, slots=torch.tensor(at, device="cuda", dtype=torch.int32))
    ofrl.delta_step(ctx, *x, small, out_small)
    torch.cuda.synchronize()
    assert torch.equal(out, out_small) and torch.equal(state[at], small)
    assert int((state.flatten(1).abs().amax(1) > 0).sum()) == 3
    ctx.close()
