"""One-token steps: states go back into their own buffer or into one that shares nothing with it."""
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
