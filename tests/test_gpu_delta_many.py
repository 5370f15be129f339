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


def test_captured_after_copies_and_other_streams():
    """Calls captured behind a copy, a fill and another stream's work give what direct calls give."""
    import torch
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    gen = torch.Generator(device="cuda").manual_seed(5)
    new = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    n, heads, dim = 200, 2, 64
    ctx = ofrl.DeltaRule(heads, heads, dim, dim, "fp32", max_tokens=n, max_episodes=2)
    ends = torch.tensor([70, n], device="cuda", dtype=torch.int32)
    src = [new(n, heads, dim) / 8, new(n, heads, dim) / 8, new(n, heads, dim), -new(n, heads).abs(), new(n, heads).sigmoid()]
    x = [torch.zeros_like(t) for t in src]
    dout, out, state = new(n, heads, dim), torch.empty(n, heads, dim, device="cuda"), new(n, heads, dim, dim)
    acted = torch.empty(n, heads, dim, device="cuda")
    grads = [torch.empty_like(t) for t in src]
    saved, norm = ctx.saved(n, 2), torch.zeros(1, device="cuda")
    lists = [ofrl.TensorList([t]) for t in (grads[0], new(1 << 19))]
    host = [t.cpu().pin_memory() for t in src]
    other = torch.cuda.Stream()

    def step():
        other.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(other):
            for a, b in zip(x[:3], host[:3]):
                a.copy_(b, non_blocking=True)
        for a, b in zip(x[3:], host[3:]):
            a.copy_(b, non_blocking=True)
        torch.cuda.current_stream().wait_stream(other)
        ofrl.delta_forward(ctx, *x, ends, out, saved=saved)
        for t in grads:
            t.zero_()
        ofrl.delta_backward(ctx, *x, ends, saved, dout, *grads)
        norm.zero_()
        ofrl.global_norm(lists[0], norm)
        state.copy_(init)
        ofrl.delta_step(ctx, *x, state, acted)
        for t in lists[1].tensors:
            t.copy_(large)
        ofrl.global_norm_clip(lists[1], 1.0, norm2)
        return [out, *grads, norm, state, acted, *lists[1].tensors, norm2]

    init, large, norm2 = state.clone(), lists[1].tensors[0].clone(), torch.zeros(1, device="cuda")
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        want = [t.clone() for t in step()]
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = step()
        for t in got:
            t.fill_(float("nan"))
        for a in x:
            a.zero_()
        for _ in range(3):
            graph.replay()
        stream.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    ctx.close()
