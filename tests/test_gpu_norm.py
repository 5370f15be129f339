"""GPU parity of the global norm over many tensors and of clipping by it."""
import math

import numpy as np
import pytest
import torch

from _gpu import need_gpu

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
# a thread's plain fp32 sum has at most 64 squares (2^-24 each step, errors of both signs), the rest is carried exactly
NORM_BOUND = 2.0 ** -20
SIZES = [[1], [0, 3], [8191, 8192, 8193], [100003], [5, 0, 17, 40000, 1, 255], list(range(1, 300)), [3_000_001, 7]]


def _tensors(sizes, dtypes, scale, seed=0, gap=0):
    """Views of one buffer per type, `gap` elements apart, so most start off a 16-byte boundary."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        dt = dtypes[i % len(dtypes)]
        buf = torch.randn(n + gap + 1, generator=g, device="cuda").mul_(scale).to(dt)
        out.append(buf[gap:gap + n] if gap else buf[:n])
    return out


def _norm(ts):
    return math.sqrt(sum(float(t.double().square().sum()) for t in ts))


@pytest.mark.parametrize("dtypes", [(F32,), (BF16,), (F32, BF16)])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("gap", [0, 1, 3])
def test_norm_and_clip(dtypes, sizes, gap):
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    ts = _tensors(sizes, dtypes, 0.7, gap=gap)
    want = _norm(ts)
    outs = _tensors(sizes, dtypes, 1.0, seed=1, gap=(gap * 2) % 5)
    lists = ofrl.TensorList(ts), ofrl.TensorList(outs)
    norm = torch.full((1,), float("nan"), device="cuda")
    ofrl.global_norm(lists[0], norm)
    assert abs(norm.item() - want) <= NORM_BOUND * want
    for limit in (want / 3, want * 3, math.inf):
        s = np.float32(limit) / np.float32(norm.item()) if norm.item() > np.float32(limit) else 1.0
        ofrl.global_norm_clip(lists[0], limit, norm, out=lists[1])
        assert abs(norm.item() - want) <= NORM_BOUND * want
        for a, b in zip(ts, outs):
            ref = a.double() * float(s)
            # the factor's division and the product round once each, then the type does
            bound = 2.0 ** -22 + (2.0 ** -8 if a.dtype == BF16 else 0.0)
            assert ((b.double() - ref).abs() <= bound * ref.abs() + 1e-38).all()
    copies = [t.clone() for t in ts]
    ofrl.global_norm_clip(lists[0], want / 3, norm)     # in place
    s = np.float32(want / 3) / np.float32(norm.item())
    for a, b in zip(copies, ts):
        ref = a.double() * float(s)
        assert ((b.double() - ref).abs() <= (2.0 ** -22 + (2.0 ** -8 if a.dtype == BF16 else 0.0)) * ref.abs() + 1e-38).all()


def test_neighbours_stay():
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    for dt in (F32, BF16):
        buf = torch.full((20000,), 2.0, device="cuda", dtype=dt)
        src = [torch.ones(n, device="cuda", dtype=dt) for n in (9001, 3, 8192)]
        outs = [buf[1:9002], buf[9005:9008], buf[9011:17203]]
        ofrl.global_norm_clip(ofrl.TensorList(src), 1.0, torch.empty(1, device="cuda"), out=ofrl.TensorList(outs))
        keep = torch.ones(20000, dtype=torch.bool, device="cuda")
        keep[1:9002] = keep[9005:9008] = keep[9011:17203] = False
        assert (buf[keep] == 2.0).all() and (buf[~keep] < 1.0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_elements(bad):
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    ts = _tensors([10000, 33], (F32,), 1.0)
    ts[1][7] = bad
    norm, outs = torch.empty(1, device="cuda"), [torch.empty_like(t) for t in ts]
    ofrl.global_norm_clip(ofrl.TensorList(ts), 1.0, norm, out=ofrl.TensorList(outs))
    if math.isnan(bad):       # a NaN norm is above nothing: the factor is 1
        assert math.isnan(norm.item())
        for a, b in zip(ts, outs):
            torch.testing.assert_close(a, b, rtol=0, atol=0, equal_nan=True)
    else:                     # max_norm / inf = 0
        assert math.isinf(norm.item())
        assert (outs[0] == 0).all() and torch.isnan(outs[1][7])


def test_zero_gradients_and_empty_lists():
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    norm = torch.full((1,), float("nan"), device="cuda")
    zero = torch.zeros(5000, device="cuda")
    ofrl.global_norm_clip(ofrl.TensorList([zero]), 1e-30, norm)
    assert norm.item() == 0.0 and (zero == 0).all()
    ofrl.global_norm_clip(ofrl.TensorList([zero[:0], zero[:0]]), 1.0, norm)
    assert norm.item() == 0.0


def test_small_and_large_elements():
    """Elements whose squares stay normal fp32 numbers, 2^-60 to 2^60."""
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    for e in (-60, 60):
        ts = _tensors([70000, 5], (F32,), 2.0 ** e)
        norm = torch.empty(1, device="cuda")
        ofrl.global_norm(ofrl.TensorList(ts), norm)
        assert abs(norm.item() - _norm(ts)) <= NORM_BOUND * _norm(ts)


def test_same_bits_each_time_and_other_streams():
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    ts = _tensors(list(range(1000, 1200)), (F32, BF16), 1.0)
    lst = ofrl.TensorList(ts)
    norm = torch.empty(1, device="cuda")
    ofrl.global_norm(lst, norm)
    first = norm.item()
    s = torch.cuda.Stream()
    for stream in (None, s, None):
        norm.fill_(-1)
        torch.cuda.synchronize()
        ofrl.global_norm(lst, norm, stream=stream)
        torch.cuda.synchronize()
        assert norm.item() == first


def test_norm_feeds_adam():
    """adam_step on each of several tensors with the global norm equals adam_step on their concatenation."""
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    ctx = ofrl.Context(8, 64, 4, max_batch=1)
    sizes = [1000, 17, 4096]
    ps, gs = _tensors(sizes, (F32,), 1.0), _tensors(sizes, (F32,), 5.0, seed=1)
    opt = ofrl.Opt(lr=1e-2, max_grad_norm=1.0)
    whole = torch.cat(ps)
    ofrl.adam_step(ctx, whole, torch.cat(gs), torch.zeros_like(whole), torch.zeros_like(whole), 1, opt)
    norm = torch.empty(1, device="cuda")
    ofrl.global_norm(ofrl.TensorList(gs), norm)
    for p, g in zip(ps, gs):
        p0 = p.clone()
        ofrl.adam_step(ctx, p0, g.contiguous(), torch.zeros_like(p0), torch.zeros_like(p0), 1, opt, grad_norm=norm)
        p.copy_(p0)
    # the two norms may differ in their last bits; Adam's first step moves by lr g / (|g| + eps)
    torch.testing.assert_close(torch.cat(ps), whole, rtol=1e-6, atol=1e-7)
    ctx.close()


def test_refusals():
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    x = torch.ones(100, device="cuda")
    norm = torch.empty(1, device="cuda")
    lst = ofrl.TensorList([x])
    with pytest.raises(ofrl.OfrlError):
        ofrl.TensorList([])
    with pytest.raises(TypeError):
        ofrl.TensorList([x.cpu()])
    with pytest.raises(TypeError):
        ofrl.TensorList([x.double()])
    with pytest.raises(ValueError):
        ofrl.TensorList([x[::2]])
    for limit in (0.0, -1.0, float("nan")):
        with pytest.raises(ofrl.OfrlError):
            ofrl.global_norm_clip(lst, limit, norm)
    with pytest.raises(ofrl.OfrlError):
        ofrl.global_norm_clip(lst, 1.0, norm, out=ofrl.TensorList([x[:99]]))
    with pytest.raises(ofrl.OfrlError):
        ofrl.global_norm_clip(lst, 1.0, norm, out=ofrl.TensorList([x.bfloat16()]))
    with pytest.raises(TypeError):
        ofrl.global_norm(lst, norm.double())
    with pytest.raises(ValueError):
        ofrl.global_norm(lst, torch.empty(2, device="cuda"))
