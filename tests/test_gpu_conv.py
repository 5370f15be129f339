"""GPU parity of the short causal convolution (forward, gradients, one token) against the fp64 definition."""
import numpy as np
import pytest
import torch

from _block import DT, ROUNDED, ROW, SUM, check, conv_inputs, dev, ends_of, host, junk, strided
from _gpu import need_gpu
from oracle import block

pytestmark = pytest.mark.gpu

LENGTHS = {"one": [1], "short": [1, 2, 3, 4, 5], "empty": [0, 3, 0, 0, 1, 2, 0], "mixed": [70, 1, 1, 33, 2, 129, 8],
           "long": [1000], "ones": [1] * 77, "ragged": [int(x) for x in np.random.default_rng(1).integers(0, 40, 60)]}


def _run(d, lengths, dtype, act, states=True, bias=True, grads=True, slices=False, ctx=None):
    import offline_rl_step_gb300 as ofrl
    t, c = d["x"].shape
    k, n = d["w"].shape[1], len(lengths)
    own = ctx is None
    if own:
        ctx = ofrl.CausalConv(c, k, act, dtype, max_tokens=t, max_episodes=n)
    x, dout, out, dx = dev(d["x"], dtype), dev(d["dout"], dtype), junk(t, c, dtype=dtype), junk(t, c, dtype=dtype)
    if slices:
        (x, dout), _ = strided([x, dout])
        (out, dx), wide = strided([out, dx])
        rest = wide[:, 2 * c:]
    w, b = dev(d["w"]), dev(d["bias"]) if bias else None
    ends = torch.from_numpy(ends_of(lengths)).cuda()
    init, final = (dev(d["init"], dtype), junk(n, c, k - 1, dtype=dtype)) if states else (None, None)
    ofrl.conv_forward(ctx, x, w, ends, out, bias=b, init_state=init, final_state=final)
    res = [out, final]
    if grads:
        dw, db = junk(c, k), junk(c) if bias else None
        dfin, dinit = (dev(d["d_final"], dtype), junk(n, c, k - 1)) if states else (None, None)
        ofrl.conv_backward(ctx, x, w, ends, dout, dx, dw, bias=b, dbias=db, init_state=init, d_final=dfin, d_init=dinit)
        res += [dx, dw, db, dinit]
    torch.cuda.synchronize()
    if slices:
        assert (rest == 0).all()
    assert ctx.poll_status()["bad_index"] == 0
    if own:
        ctx.close()
    return [host(r) for r in res]


def _check(d, lengths, dtype, act, got, states=True, bias=True):
    ends, b, init = ends_of(lengths), d["bias"] if bias else None, d["init"] if states else None
    out, final, _ = block.conv_forward(d["x"], d["w"], b, ends, act, init)
    rounded = ROUNDED[dtype]
    check(got[0], out, ROW + rounded, "out")
    if states:
        assert (got[1] == final).all()      # copies of inputs
    if len(got) > 2:
        dx, dw, db, dinit = block.conv_backward(d["x"], d["w"], b, ends, d["dout"], act, init,
                                                d["d_final"] if states else None)
        check(got[2], dx, ROW + rounded, "dx")
        check(got[3], dw, SUM, "dw")
        if bias:
            check(got[4], db, SUM, "dbias")
        if states:
            check(got[5], dinit, ROW, "d_init")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("lengths", list(LENGTHS), ids=str)
def test_parity(dtype, width, lengths):
    need_gpu()
    ln = LENGTHS[lengths]
    for c, act, states, bias, slices in ((8, "silu", True, True, False), (136, "none", True, False, True),
                                         (360, "silu", False, True, True)):
        d = conv_inputs(ln, c, width, c + width, dtype)
        got = _run(d, ln, dtype, act, states, bias, slices=slices)
        _check(d, ln, dtype, act, got, states, bias)


def test_many_tokens_and_channels():
    """Runs of every length, several CTAs along both axes."""
    need_gpu()
    for t, c in ((20000, 136), (3000, 1040), (60000, 24)):
        lengths = [t // 3, 0, t - t // 3 - 1, 1]
        d = conv_inputs(lengths, c, 4, 3, "bf16")
        _check(d, lengths, "bf16", "silu", _run(d, lengths, "bf16", "silu"))


def test_tokens_behind_the_last_episode_stay():
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    d = conv_inputs([50], 16, 4, 0, "fp32")
    ctx = ofrl.CausalConv(16, 4, "silu", "fp32", 50, 3)
    ends = torch.tensor([10, 30, 30], dtype=torch.int32, device="cuda")
    x, w, dout = dev(d["x"]), dev(d["w"]), dev(d["dout"])
    x[30:], dout[30:] = float("nan"), float("nan")
    out, dx, dw = (torch.full_like(x, 7.0), torch.full_like(x, 7.0), junk(16, 4))
    ofrl.conv_forward(ctx, x, w, ends, out)
    ofrl.conv_backward(ctx, x, w, ends, dout, dx, dw)
    assert (out[30:] == 7).all() and (dx[30:] == 7).all()
    want, _, _ = block.conv_forward(d["x"][:30], d["w"], None, [10, 30, 30], "silu")
    check(host(out[:30]), want, ROW, "out")
    gx, gw, _, _ = block.conv_backward(d["x"][:30], d["w"], None, [10, 30, 30], d["dout"][:30], "silu")
    check(host(dx[:30]), gx, ROW, "dx")
    check(host(dw), gw, SUM, "dw")


def test_no_tokens():
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    for n in (0, 3):
        ctx = ofrl.CausalConv(16, 3, "silu", "bf16", 0, n)
        x = torch.empty(0, 16, device="cuda", dtype=torch.bfloat16)
        ends = torch.zeros(n, dtype=torch.int32, device="cuda")
        init = torch.randn(n, 16, 2, device="cuda").bfloat16()
        final, dinit, dw, db = torch.zeros_like(init), junk(n, 16, 2), junk(16, 3), junk(16)
        ofrl.conv_forward(ctx, x, torch.ones(16, 3, device="cuda"), ends, x.clone(), init_state=init, final_state=final)
        ofrl.conv_backward(ctx, x, torch.ones(16, 3, device="cuda"), ends, x, x.clone(), dw, dbias=db, init_state=init,
                           d_final=init, d_init=dinit)
        assert torch.equal(final, init) and torch.equal(dinit, init.float())
        assert (dw == 0).all() and (db == 0).all()


def test_bad_ends_are_counted():
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    ctx = ofrl.CausalConv(16, 4, "silu", "fp32", 100, 40)
    x, w = torch.randn(100, 16, device="cuda"), torch.randn(16, 4, device="cuda")
    guard = torch.full((3, 100, 16), 5.0, device="cuda")
    state = torch.zeros(4, 16, 3, device="cuda")
    for ends, bad in (([50, 40, 70, 100], 1), ([-3, 101, 20, 2 ** 30], 4), ([10, 20, 30, 2 ** 31 - 1], 1),
                      ([10, 20, 30, 100], 0)):
        e = torch.tensor(ends, dtype=torch.int32, device="cuda")
        ofrl.conv_forward(ctx, x, w, e, guard[1], init_state=state, final_state=state.clone())
        ofrl.conv_backward(ctx, x, w, e, x, guard[1], torch.empty_like(w), init_state=state, d_final=state,
                           d_init=torch.empty_like(state))
        assert ctx.poll_status()["bad_index"] == bad, ends
    assert (guard[0] == 5).all() and (guard[2] == 5).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_inputs_stay(bad):
    """A token that is not finite reaches its channel, the tokens that take it, and its episode."""
    need_gpu()
    lengths = [20, 20, 20]
    d = conv_inputs(lengths, 16, 4, 4, "fp32")
    clean = _run(d, lengths, "fp32", "silu")
    d["x"][25, 3] = bad
    got = _run(d, lengths, "fp32", "silu")
    touched = np.zeros((60, 16), bool)
    touched[25:29, 3] = True
    assert (np.isfinite(got[0]) == ~touched).all() if bad != np.inf else np.isfinite(got[0][~touched]).all()
    assert (got[0][~touched] == clean[0][~touched]).all()
    near = np.zeros((60, 16), bool)      # dx of tokens that share an output with it
    near[22:29, 3] = True
    assert (got[2][~near] == clean[2][~near]).all()
    assert (np.delete(got[3], 3, 0) == np.delete(clean[3], 3, 0)).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("width", [2, 3, 4])
def test_step_is_reading_one_token_at_a_time(dtype, width):
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    n, length, c = 5, 9, 24
    lengths = [length] * n
    d = conv_inputs(lengths, c, width, 9, dtype)
    want = _run(d, lengths, dtype, "silu", grads=False)
    ctx = ofrl.CausalConv(c, width, "silu", dtype, 0, 0, backward=False)
    x = dev(d["x"], dtype).view(n, length, c)
    w, b = dev(d["w"]), dev(d["bias"])
    state, other = dev(d["init"], dtype), junk(n, c, width - 1, dtype=dtype)
    outs = []
    for i in range(length):
        out = junk(n, c, dtype=dtype)
        if i % 2:      # in place and into another buffer in turn
            ofrl.conv_step(ctx, x[:, i], w, state, out, bias=b)
        else:
            ofrl.conv_step(ctx, x[:, i], w, state, out, bias=b, new_state=other)
            state, other = other, state
        outs.append(out)
    assert (host(torch.stack(outs, 1).view(n * length, c)) == want[0]).all()
    assert (host(state) == want[1]).all()


def test_step_slots():
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    c, k, slots = 16, 4, 6
    d = conv_inputs([3], c, k, 2, "fp32")
    ctx = ofrl.CausalConv(c, k, "silu", "fp32", 0, 0, backward=False)
    x, w = dev(d["x"]), dev(d["w"])
    state = torch.randn(slots, c, k - 1, device="cuda")
    before, out = state.clone(), junk(3, c)
    ofrl.conv_step(ctx, x, w, state, out, slots=torch.tensor([4, -1, 0], dtype=torch.int32, device="cuda"))
    assert ctx.poll_status()["bad_index"] == 1
    assert (out[1] == 0).all()
    for i, s in ((0, 4), (2, 0)):
        want, final, _ = block.conv_forward(d["x"][i:i + 1], d["w"], None, [1], "silu", host(before[s])[None])
        check(host(out[i]), want[0], ROW, "out")
        assert (host(state[s]) == final[0]).all()
    for s in (1, 2, 3, 5):
        assert torch.equal(state[s], before[s])
    for bad in (slots, 2 ** 31 - 1, -2 ** 31):
        ofrl.conv_step(ctx, x[:1], w, state, out[:1], slots=torch.tensor([bad], dtype=torch.int32, device="cuda"))
    assert ctx.poll_status()["bad_index"] == 3
    # many tokens a thread: more environments than the GPU holds threads
    n = 40000
    c2 = ofrl.CausalConv(128, 2, "none", "fp32", 0, 0, backward=False)
    x, w = torch.randn(n, 128, device="cuda"), torch.randn(128, 2, device="cuda")
    state, out = torch.randn(n, 128, 1, device="cuda"), junk(n, 128)
    want = state[:, :, 0].double() * w[:, 0].double() + x.double() * w[:, 1].double()
    ofrl.conv_step(c2, x, w, state, out)
    assert torch.equal(state[:, :, 0], x)
    check(host(out), want.cpu().numpy(), ROW, "out")


def test_streams_graphs_and_repeats():
    """On another stream, captured and replayed, and again: the same bits."""
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    lengths, c = [100, 0, 33, 300], 72
    d = conv_inputs(lengths, c, 4, 6, "bf16")
    want = _run(d, lengths, "bf16", "silu")
    again = _run(d, lengths, "bf16", "silu")
    assert all((a == b).all() for a, b in zip(want, again))
    ctx = ofrl.CausalConv(c, 4, "silu", "bf16", 433, 4)
    x, w, b, dout = dev(d["x"], "bf16"), dev(d["w"]), dev(d["bias"]), dev(d["dout"], "bf16")
    ends, init, dfin = torch.from_numpy(ends_of(lengths)).cuda(), dev(d["init"], "bf16"), dev(d["d_final"], "bf16")
    outs = [junk(433, c, dtype="bf16"), junk(4, c, 3, dtype="bf16"), junk(433, c, dtype="bf16"), junk(c, 4), junk(c),
            junk(4, c, 3)]

    def both():
        ofrl.conv_forward(ctx, x, w, ends, outs[0], bias=b, init_state=init, final_state=outs[1])
        ofrl.conv_backward(ctx, x, w, ends, dout, outs[2], outs[3], bias=b, dbias=outs[4], init_state=init, d_final=dfin,
                           d_init=outs[5])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.synchronize()
    assert all((host(a) == b).all() for a, b in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for _ in range(2):
        for o in outs:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all((host(a) == b).all() for a, b in zip(outs, want))


def test_refusals():
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    ctx = ofrl.CausalConv(16, 4, "silu", "bf16", 100, 4)
    x, w = torch.zeros(100, 16, device="cuda", dtype=DT["bf16"]), torch.zeros(16, 4, device="cuda")
    ends = torch.tensor([100], dtype=torch.int32, device="cuda")
    out = torch.zeros_like(x)
    wide = torch.zeros(100, 64, device="cuda", dtype=DT["bf16"])

    def refused(error, *a, **k):
        with pytest.raises(error):
            ofrl.conv_forward(ctx, *a, **k)

    refused(TypeError, x.float(), w, ends, out)
    refused(TypeError, x, w.bfloat16(), ends, out)
    refused(TypeError, x, w, ends.long(), out)
    refused(TypeError, x.cpu(), w, ends, out)
    refused(ValueError, x[:, :8], w, ends, out)
    refused(ValueError, x, w.T.contiguous(), ends, out)
    refused(ValueError, x, w, ends, out[:50])
    refused(ValueError, wide[:, ::4], w, ends, out)                      # not dense
    refused(ofrl.OfrlError, wide[:, 4:20], w, ends, out)                 # rows off 16 bytes
    refused(ofrl.OfrlError, x[:1].expand(100, 16), w, ends, out)         # rows on top of each other
    refused(ofrl.OfrlError, x, w, ends[:0], out)                         # tokens without episodes
    refused(ofrl.OfrlError, torch.zeros(101, 16, device="cuda", dtype=DT["bf16"]), w, ends,
            torch.zeros(101, 16, device="cuda", dtype=DT["bf16"]))       # more than the workspace is for
    refused(ofrl.OfrlError, x, w, torch.full((5,), 100, dtype=torch.int32, device="cuda"), out)
    refused(TypeError, x, w, ends, out, init_state=torch.zeros(1, 16, 3, device="cuda"))
    with pytest.raises(TypeError):
        ofrl.conv_backward(ctx, x, w, ends, x, out, None)
    forward_only = ofrl.CausalConv(16, 4, "silu", "bf16", 100, 4, backward=False)
    with pytest.raises(ofrl.OfrlError):
        ofrl.conv_backward(forward_only, x, w, ends, x, out, torch.zeros_like(w))
    state = torch.zeros(3, 16, 3, device="cuda", dtype=DT["bf16"])
    with pytest.raises(ofrl.OfrlError):
        ofrl.conv_step(ctx, x[:4], w, state, out[:4])                    # more tokens than slots
    ctx.close()
    with pytest.raises(ValueError, match="closed"):
        ofrl.conv_forward(ctx, x, w, ends, out)
