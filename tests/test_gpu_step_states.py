"""States go back into their own buffer or into one that shares nothing with it."""
import pytest
import torch

from _gpu import need_gpu

pytestmark = pytest.mark.gpu


def _refused_but_apart(step, shape, dtype):
    """step(state, new_state) with views of one buffer of six slots: only the shifted ones are refused, and then nothing
    is written."""
    import offline_rl_step_gb300 as ofrl
    buf = torch.randn(6, *shape, device="cuda").to(dtype)
    was = buf.clone()
    for a, b in ((0, 1), (1, 0), (0, 2), (2, 0)):
        with pytest.raises(ofrl.OfrlError):
            step(buf[a:a + 3], buf[b:b + 3])
    assert torch.equal(buf, was)
    step(buf[:3], buf[3:])
    assert torch.equal(buf[:3], was[:3]) and not torch.equal(buf[3:], was[3:])
    apart = buf[3:].clone()
    step(buf[:3], buf[:3])
    assert torch.equal(buf[:3], apart) and torch.equal(buf[3:], apart)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_scan(dtype):
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    c, n, ty = 24, 16, {"fp32": torch.float32, "bf16": torch.bfloat16}[dtype]
    ctx = ofrl.SelectiveScan(c, n, 1, dtype, True, 0, 0, backward=False)
    x, B, A, out = (torch.randn(3, c, device="cuda").to(ty), torch.randn(3, 1, n, device="cuda").to(ty),
                    -torch.ones(c, n, device="cuda"), torch.empty(3, c, device="cuda", dtype=ty))
    _refused_but_apart(lambda s, new: ofrl.scan_step(ctx, x, x, A, B, B, s, out, new_state=new), (c, n), torch.float32)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_convolution(dtype):
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    c, ty = 32, {"fp32": torch.float32, "bf16": torch.bfloat16}[dtype]
    for width in (2, 4):
        ctx = ofrl.CausalConv(c, width, "silu", dtype, 0, 0, backward=False)
        x, w = torch.randn(3, c, device="cuda").to(ty), torch.randn(c, width, device="cuda")
        out = torch.empty_like(x)
        _refused_but_apart(lambda s, new: ofrl.conv_step(ctx, x, w, s, out, new_state=new), (c, width - 1), ty)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_delta_rule(dtype):
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    ty = {"fp32": torch.float32, "bf16": torch.bfloat16}[dtype]
    for heads, dk, dv in ((2, 16, 24), (1, 64, 64)):
        ctx = ofrl.DeltaRule(heads, heads, dk, dv, dtype, max_tokens=0, max_episodes=0, backward=False)
        q, k, v = (torch.randn(3, heads, d, device="cuda").to(ty) for d in (dk, dk, dv))
        g, beta = -torch.rand(3, heads, device="cuda").to(ty), torch.rand(3, heads, device="cuda").to(ty)
        out = torch.empty_like(v)
        _refused_but_apart(lambda s, new: ofrl.delta_step(ctx, q, k, v, g, beta, s, out, new_state=new), (heads, dv, dk),
                           torch.float32)


def test_delta_rule_over_episodes():
    """The final states may take the initial ones' place, their gradients likewise."""
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    t, h, d, e = 60, 2, 16, 3
    ctx = ofrl.DeltaRule(h, h, d, d, "fp32", max_tokens=t, max_episodes=e)
    q, k, v, dout = torch.randn(4, t, h, d, device="cuda")
    g, beta = -torch.rand(t, h, device="cuda"), torch.rand(t, h, device="cuda")
    ends, out, saved = torch.tensor([20, 30, t], dtype=torch.int32, device="cuda"), torch.empty_like(v), ctx.saved(t, e)
    grads = [torch.empty_like(x) for x in (q, k, v, g, beta)]
    states = torch.randn(6, h, d, d, device="cuda")

    def forward(init, final):
        ofrl.delta_forward(ctx, q, k, v, g, beta, ends, out, init_state=init, final_state=final, saved=saved)

    def backward(init, final):      # of the final states, of the initial ones
        ofrl.delta_backward(ctx, q, k, v, g, beta, ends, saved, dout, *grads, d_final=init, d_init=final)

    for call in (forward, backward):
        was = states.clone()
        for a, b in ((0, 1), (2, 0)):
            with pytest.raises(ofrl.OfrlError):
                call(states[a:a + 3], states[b:b + 3])
        assert torch.equal(states, was)
        call(states[:3], states[3:])
        apart = states[3:].clone()
        call(states[:3], states[:3])
        assert torch.equal(states[:3], apart)
