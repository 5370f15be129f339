"""GPU parity of the gated delta rule (forward, backward, one step) against the fp64 recurrence."""
import numpy as np
import pytest
import torch

from _delta import BOUND, STATE_BOUND, U, bf16, check, ends_of, inputs
from _gpu import need_gpu
from oracle import delta

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
ROUND = {"fp32": lambda x: x, "bf16": bf16}
NAMES = ("q", "k", "v", "g", "beta")


def _dev(x, dtype="fp32"):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda().to(DT[dtype])


def _host(t):
    return t.double().cpu().numpy()


def _run(d, lengths, dtype, scale=0.3, states=True, grads=True, strided=False, ctx=None, junk=float("nan")):
    """out, final, (dq, dk, dv, dg, dbeta, d_init) of the library; every output starts as `junk`."""
    import offline_rl_step_gb300 as ofrl
    t, hk, dk = d["q"].shape
    hv, dv = d["v"].shape[1:]
    n = len(lengths)
    own = ctx is None
    if own:
        ctx = ofrl.DeltaRule(hk, hv, dk, dv, dtype, max_tokens=t, max_episodes=n)
    x = [_dev(d[name], dtype) for name in NAMES]
    new = lambda *s: torch.full(s, junk, device="cuda", dtype=DT[dtype])
    gr = [new(*y.shape) for y in x]
    if strided:      # q, k, v as slices of one projection, the gates of another; gradients likewise
        def fuse(parts):
            return torch.cat([p.flatten(1) for p in parts], 1).split([p[0].numel() for p in parts], 1)
        shapes = [y.shape[1:] for y in x]
        pad = _dev(np.zeros((t, 8)), dtype)
        x = [y.unflatten(1, s) for y, s in zip(fuse(x[:3] + [pad])[:3] + fuse(x[3:] + [pad[:, :3]])[:2], shapes)]
        gr = [y.unflatten(1, s) for y, s in zip(fuse(gr[:3] + [pad])[:3] + fuse(gr[3:] + [pad[:, :3]])[:2], shapes)]
    ends = torch.from_numpy(ends_of(lengths)).cuda()
    out = new(t, hv, dv)
    f32 = lambda: torch.full((n, hv, dv, dk), junk, device="cuda")
    init, final = (_dev(d["init"]), f32()) if states else (None, None)
    saved = ctx.saved(t, n).fill_(0xFF) if grads else None
    ofrl.delta_forward(ctx, *x, ends, out, scale=scale, init_state=init, final_state=final, saved=saved)
    res = [out, final]
    if grads:
        dfin, dinit = (_dev(d["d_final"]), f32()) if states else (None, None)
        ofrl.delta_backward(ctx, *x, ends, saved, _dev(d["dout"], dtype), *gr, scale=scale, d_final=dfin,
                            d_init=dinit)
        res += [*gr, dinit]
    torch.cuda.synchronize()
    assert ctx.poll_status()["bad_index"] == 0
    if own:
        ctx.close()
    return [None if r is None else _host(r) for r in res]


def _want(d, lengths, scale=0.3, states=True):
    a = [d[n] for n in NAMES]
    init, dfin = (d["init"], d["d_final"]) if states else (None, None)
    out, final = delta.forward(*a, ends_of(lengths), scale, init=init)
    return [out, final, *delta.backward(*a, ends_of(lengths), scale, d["dout"], init=init, d_final=dfin)]


LABELS = ("out", "final", "dq", "dk", "dv", "dg", "dbeta", "d_init")


def _compare(got, want, dtype, factor=1.0):
    for name, x, y in zip(LABELS, got, want):
        if x is not None:
            check(x, y, factor * (STATE_BOUND if name in ("final", "d_init") and dtype == "fp32" else
                                  GRAD_STATE_BOUND if name == "d_init" else STATE_BOUND if name == "final" else
                                  BOUND[dtype]), name)


# with bf16 tokens the gradient of the initial state passes through operands of 11 significand bits
GRAD_STATE_BOUND = 2e-3

RAGGED = [5, 64, 0, 1, 65, 130, 63, 2, 128]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("hk,hv,dk,dv", [(1, 1, 64, 64), (2, 4, 128, 128), (1, 3, 40, 72), (2, 2, 8, 8),
                                         (1, 2, 128, 64), (1, 1, 64, 128), (3, 3, 120, 16), (1, 1, 16, 104)])
def test_forward_and_backward(dtype, hk, hv, dk, dv):
    need_gpu()
    d = inputs(RAGGED, hk, hv, dk, dv, seed=dk + dv, rnd=ROUND[dtype])
    _compare(_run(d, RAGGED, dtype), _want(d, RAGGED), dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("lengths", [[1], [64], [65], [0, 0, 3, 0], [1] * 40, [700]])
def test_lengths(dtype, lengths):
    need_gpu()
    d = inputs(lengths, 1, 2, 64, 64, seed=len(lengths), rnd=ROUND[dtype])
    _compare(_run(d, lengths, dtype), _want(d, lengths), dtype)
    _compare(_run(d, lengths, dtype, states=False), _want(d, lengths, states=False), dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("hk,hv,dk,dv", [(1, 2, 64, 64), (2, 2, 24, 48), (1, 1, 128, 128)])
def test_slices_of_a_fused_projection(dtype, hk, hv, dk, dv):
    need_gpu()
    lengths = [70, 3, 129]
    d = inputs(lengths, hk, hv, dk, dv, seed=3, rnd=ROUND[dtype])
    for a, b in zip(_run(d, lengths, dtype, strided=True), _run(d, lengths, dtype)):
        np.testing.assert_array_equal(a, b)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_forward_without_backward_gives_the_same_outputs(dtype):
    need_gpu()
    d = inputs(RAGGED, 2, 4, 64, 64, seed=9, rnd=ROUND[dtype])
    alone, both = _run(d, RAGGED, dtype, grads=False), _run(d, RAGGED, dtype)
    want = _want(d, RAGGED)
    check(alone[0], want[0], BOUND[dtype], "out")
    check(alone[1], want[1], STATE_BOUND, "final")
    check(both[0], alone[0], BOUND[dtype], "out with and without saved states")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_forgetting_no_strength_and_zero_keys(dtype):
    """g = -inf at, before and after chunk borders; tokens of no strength; zero keys and queries; strong decay."""
    need_gpu()
    lengths = [200, 66]
    d = inputs(lengths, 1, 2, 64, 64, seed=11, decay=20.0, rnd=ROUND[dtype])
    for t in (0, 1, 63, 64, 65, 127, 128, 199, 200, 263):
        d["g"][t, t % 2] = -np.inf
    d["beta"][10:40, 0] = 0.0
    d["k"][50:60] = 0.0
    d["q"][55:70] = 0.0
    d["k"][128:192] = 0.0     # a whole chunk
    d["dout"][210:] = 0.0
    _compare(_run(d, lengths, dtype), _want(d, lengths), dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("kq,vv,dd", [(2.0 ** 12, 1.0, 1.0), (2.0 ** -14, 2.0 ** 20, 2.0 ** -24), (1.0, 2.0 ** -20, 2.0 ** 18)])
def test_magnitudes(dtype, kq, vv, dd):
    """Keys, values and gradients far from 1 (beta scaled so that beta |k|^2 stays in (0, 1))."""
    need_gpu()
    lengths = [130, 40]
    d = inputs(lengths, 1, 2, 64, 64, seed=13, rnd=ROUND[dtype])
    for name, f in (("q", kq), ("k", kq), ("beta", kq ** -2), ("v", vv), ("dout", dd), ("init", vv / kq),
                    ("d_final", dd * kq)):
        d[name] = (d[name] * np.float32(f)).astype(np.float32)     # powers of two: exact
    _compare(_run(d, lengths, dtype), _want(d, lengths), dtype)


def test_rows_of_very_different_size():
    """Within a chunk, keys, values and output gradients whose sizes spread over four decades."""
    need_gpu()
    lengths = [150]
    d = inputs(lengths, 1, 1, 64, 64, seed=17, rnd=bf16)
    f = np.exp2(np.random.default_rng(0).integers(-13, 1, (150, 1, 1))).astype(np.float32)
    for name, x in (("k", f), ("v", f[::-1]), ("dout", np.roll(f, 7))):
        d[name] = d[name] * x
    _compare(_run(d, lengths, "bf16"), _want(d, lengths), "bf16")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_same_call_same_bits_and_no_trace_of_other_calls(dtype):
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    d = inputs(RAGGED, 1, 2, 64, 64, seed=21, rnd=ROUND[dtype])
    o = inputs([300, 11], 1, 2, 64, 64, seed=22, rnd=ROUND[dtype])
    ctx = ofrl.DeltaRule(1, 2, 64, 64, dtype, max_tokens=1000, max_episodes=20)
    first = _run(d, RAGGED, dtype, ctx=ctx)
    _run(o, [300, 11], dtype, ctx=ctx)
    for a, b in zip(first, _run(d, RAGGED, dtype, ctx=ctx, junk=7.0)):
        np.testing.assert_array_equal(a, b)
    ctx.close()


def test_carrying_the_state_over_two_calls():
    need_gpu()
    d = inputs([300], 1, 2, 64, 64, seed=23)
    whole = _run(d, [300], "fp32", grads=False)
    a = {n: x[:130] if n in NAMES else x for n, x in d.items()}
    first = _run(a, [130], "fp32", grads=False)
    b = {n: x[130:] if n in NAMES else x for n, x in d.items()}
    b["init"] = first[1].astype(np.float32)
    second = _run(b, [170], "fp32", grads=False)
    check(np.concatenate([first[0], second[0]]), whole[0], 2 * BOUND["fp32"], "out")
    check(second[1], whole[1], 2 * STATE_BOUND, "final")


def test_final_state_may_be_the_initial_one_and_tokens_past_the_last_end_stay():
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    lengths = [70, 5]
    d = inputs([70, 5, 9], 1, 1, 64, 64, seed=25)
    want = _run({n: x[:75] if n in NAMES else x[:2] for n, x in d.items() if n != "dout"}, lengths, "fp32",
                grads=False)
    ctx = ofrl.DeltaRule(1, 1, 64, 64, "fp32", max_tokens=84, max_episodes=2, backward=False)
    state, out = _dev(d["init"][:2]), torch.full((84, 1, 64), 7.0, device="cuda")
    ofrl.delta_forward(ctx, *[_dev(d[n]) for n in NAMES], torch.from_numpy(ends_of(lengths)).cuda(), out, scale=0.3,
                       init_state=state, final_state=state)
    np.testing.assert_array_equal(_host(out[:75]), want[0])
    np.testing.assert_array_equal(_host(state), want[1])
    assert (out[75:] == 7.0).all()
    ctx.close()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("lengths,hk,hv,dk,dv", [([3000], 1, 2, 64, 64), ([2000, 0, 70, 1500], 1, 1, 128, 128),
                                                 ([1000], 1, 1, 40, 104), ([5001], 2, 2, 128, 24)])
def test_long_episodes(dtype, lengths, hk, hv, dk, dv):
    """Few heads and long episodes: read in parts, with the states in one buffer that is replaced."""
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    d = inputs(lengths, hk, hv, dk, dv, seed=37, rnd=ROUND[dtype])
    t, n = sum(lengths), len(lengths)
    out, final = delta.forward(*[d[x] for x in NAMES], ends_of(lengths), 0.3, init=d["init"])
    ctx = ofrl.DeltaRule(hk, hv, dk, dv, dtype, max_tokens=t, max_episodes=n, backward=False)
    x, ends = [_dev(d[name], dtype) for name in NAMES], torch.from_numpy(ends_of(lengths)).cuda()
    got = torch.full((t, hv, dv), float("nan"), device="cuda", dtype=DT[dtype])
    state = _dev(d["init"])
    ofrl.delta_forward(ctx, *x, ends, got, scale=0.3, init_state=state, final_state=state)
    check(_host(got), out, BOUND[dtype], "out")
    check(_host(state), final, STATE_BOUND, "final")
    ofrl.delta_forward(ctx, *x, ends, got, scale=0.3, init_state=_dev(d["init"]))
    check(_host(got), out, BOUND[dtype], "out alone")
    ctx.close()


def test_another_stream():
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    d = inputs(RAGGED, 1, 2, 64, 64, seed=27)
    want = _run(d, RAGGED, "fp32", grads=False)
    ctx = ofrl.DeltaRule(1, 2, 64, 64, "fp32", max_tokens=500, max_episodes=20, backward=False)
    x, ends = [_dev(d[n]) for n in NAMES], torch.from_numpy(ends_of(RAGGED)).cuda()
    out = torch.empty(int(sum(RAGGED)), 2, 64, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ofrl.delta_forward(ctx, *x, ends, out, scale=0.3, init_state=_dev(d["init"]), stream=s)
    s.synchronize()
    np.testing.assert_array_equal(_host(out), want[0])
    ctx.close()


def test_bad_ends_are_counted():
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    d = inputs([100], 1, 1, 64, 64, seed=29)
    ctx = ofrl.DeltaRule(1, 1, 64, 64, "fp32", max_tokens=100, max_episodes=8, backward=False)
    out = torch.zeros(100, 1, 64, device="cuda")
    for ends, bad in (([40, 20, 100], 1), ([40, 101], 1), ([-5, 100], 1), ([10, 100, 100], 0), ([0, 100], 0)):
        ofrl.delta_forward(ctx, *[_dev(d[n]) for n in NAMES], torch.tensor(ends, dtype=torch.int32, device="cuda"), out)
        assert ctx.poll_status()["bad_index"] == bad, ends
    ctx.close()


# ---- one token --------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("n,hk,hv,dk,dv", [(1, 2, 2, 64, 64), (7, 1, 3, 40, 72), (300, 2, 4, 128, 128), (5, 1, 1, 8, 8),
                                           (33, 1, 1, 128, 24), (1000, 1, 2, 24, 128)])
def test_step(dtype, n, hk, hv, dk, dv):
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    lengths = [1] * n
    d = inputs(lengths, hk, hv, dk, dv, seed=n, rnd=ROUND[dtype])
    d["g"][n // 2] = -np.inf
    out, final = delta.forward(*[d[x] for x in NAMES], ends_of(lengths), 0.3, init=d["init"])
    ctx = ofrl.DeltaRule(hk, hv, dk, dv, dtype, max_tokens=0, max_episodes=0, backward=False)
    x = [_dev(d[name], dtype) for name in NAMES]
    state, new = _dev(d["init"]), torch.full((n, hv, dv, dk), float("nan"), device="cuda")
    got = torch.full((n, hv, dv), float("nan"), device="cuda", dtype=DT[dtype])
    # one product and sum in fp32 over at most 128 terms, then the output's rounding
    bound = 2.0 ** -24 * 16 + U[dtype]
    ofrl.delta_step(ctx, *x, state, got, scale=0.3, new_state=new)
    check(_host(got), out, bound, "out")
    check(_host(new), final, 2.0 ** -20, "state")
    np.testing.assert_array_equal(_host(state), d["init"])
    ofrl.delta_step(ctx, *x, state, got, scale=0.3)
    check(_host(got), out, bound, "out in place")
    np.testing.assert_array_equal(_host(state), _host(new))
    ctx.close()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_step_slots(dtype):
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    n, slots = 6, [3, -1, 9, 0, 10, 7]
    d = inputs([1] * n, 1, 2, 64, 40, seed=2, rnd=ROUND[dtype])
    pool = np.random.default_rng(3).standard_normal((10, 2, 40, 64)).astype(np.float32)
    ctx = ofrl.DeltaRule(1, 2, 64, 40, dtype, max_tokens=0, max_episodes=0, backward=False)
    state, out = _dev(pool), torch.full((n, 2, 40), 7.0, device="cuda", dtype=DT[dtype])
    ofrl.delta_step(ctx, *[_dev(d[x], dtype) for x in NAMES], state, out, scale=0.3,
                    slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    assert ctx.poll_status()["bad_index"] == 2
    want = pool.astype(np.float64)
    for i, s in enumerate(slots):
        if not 0 <= s < 10:
            assert (out[i] == 0).all()
            continue
        o, f = delta.forward(*[d[x][i:i + 1] for x in NAMES], [1], 0.3, init=pool[s:s + 1])
        check(_host(out[i]), ROUND[dtype](o[0].astype(np.float32)), 2.0 ** -20 + U[dtype], f"out {i}")
        want[s] = f[0]
    check(_host(state), want, 2.0 ** -20, "states")
    ctx.close()


def test_stepping_follows_reading():
    """Acting on from the state that a forward call left gives what one longer forward call gives."""
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    lengths = [75, 75, 75]
    d = inputs(lengths, 1, 2, 64, 64, seed=31)
    out, final = delta.forward(*[d[x] for x in NAMES], ends_of(lengths), 0.3)
    ctx = ofrl.DeltaRule(1, 2, 64, 64, "fp32", max_tokens=225, max_episodes=3, backward=False)
    x = {n: _dev(d[n]).unflatten(0, (3, 75)) for n in NAMES}
    state, got = torch.empty(3, 2, 64, 64, device="cuda"), torch.empty(210, 2, 64, device="cuda")
    ofrl.delta_forward(ctx, *[x[n][:, :70].flatten(0, 1) for n in NAMES], torch.from_numpy(ends_of([70] * 3)).cuda(),
                       got, scale=0.3, final_state=state)
    for t in range(70, 75):
        o = torch.empty(3, 2, 64, device="cuda")
        ofrl.delta_step(ctx, *[x[n][:, t] for n in NAMES], state, o, scale=0.3)
        check(_host(o), out.reshape(3, 75, 2, 64)[:, t], BOUND["fp32"], f"token {t}")
    check(_host(state), final, STATE_BOUND, "final")
    ctx.close()


# ---- gradients against differences of the forward kernel ----------------------------------------------------------


def test_gradients_against_differences_of_the_forward():
    """Along random directions: (f(x + h d) - f(x - h d)) / 2h with fp32 outputs summed in fp64.  Truncation is
    O(h^2) and the outputs' error (1e-5 of their norm, random over 1e4 of them) over h = 1/64 stays below 1e-3."""
    need_gpu()
    lengths = [150, 20]
    d = inputs(lengths, 1, 2, 64, 64, seed=33)
    got = _run(d, lengths, "fp32")
    r = np.random.default_rng(1)
    h = 2.0 ** -6
    for name, grad in zip(NAMES + ("init",), got[2:]):
        step = r.standard_normal(d[name].shape) * (np.abs(d[name]) if name in ("g", "beta") else 1.0)
        step *= np.linalg.norm(d[name]) / np.linalg.norm(step)

        def loss(sign):
            x = dict(d)
            x[name] = (d[name] + sign * h * step).astype(np.float32)
            o = _run(x, lengths, "fp32", grads=False)
            return (o[0] * d["dout"]).sum() + (o[1] * d["d_final"]).sum(), x[name].astype(np.float64)

        (hi, xh), (lo, xl) = loss(1), loss(-1)
        slope = ((xh - xl) * grad).sum()
        size = np.linalg.norm(grad) * np.linalg.norm(xh - xl) / np.sqrt(grad.size)
        assert abs((hi - lo) - slope) <= 2e-2 * max(abs(slope), 10 * size), (name, hi - lo, slope, size)


# ---- refusals -------------------------------------------------------------------------------------------------------


def test_refusals():
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    d = inputs([70], 1, 2, 64, 64, seed=35)
    ctx = ofrl.DeltaRule(1, 2, 64, 64, "fp32", max_tokens=70, max_episodes=1, backward=False)
    x, ends = [_dev(d[n]) for n in NAMES], torch.tensor([70], dtype=torch.int32, device="cuda")
    out = torch.empty(70, 2, 64, device="cuda")
    bad = [
        (TypeError, [x[0].cpu(), *x[1:], ends, out]), (TypeError, [x[0].bfloat16(), *x[1:], ends, out]),
        (ValueError, [x[0][:, :, :32], *x[1:], ends, out]), (ValueError, [x[0][:69], *x[1:], ends, out]),
        (ValueError, [*x[:2], x[2].transpose(1, 2).contiguous().transpose(1, 2), *x[3:], ends, out]),
        (TypeError, [*x, ends.long(), out]), (ValueError, [*x, ends, out[:, :1]]),
        (ofrl.OfrlError, [*x, ends.repeat(2), out]),                        # more episodes than the context holds
        (ofrl.OfrlError, [torch.empty(70 * 64 + 1, device="cuda")[1:].view(70, 1, 64), *x[1:], ends, out]),
    ]
    for err, args in bad:
        with pytest.raises(err):
            ofrl.delta_forward(ctx, *args)
    with pytest.raises(ofrl.OfrlError):
        ofrl.delta_forward(ctx, *x, ends, out, scale=float("nan"))
    with pytest.raises(ValueError):
        ofrl.delta_forward(ctx, *x, ends, out, init_state=torch.zeros(2, 2, 64, 64, device="cuda"))
    with pytest.raises(ValueError):
        ofrl.delta_forward(ctx, *x, ends, out, saved=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ofrl.OfrlError):       # a context without room for gradients
        ofrl.delta_backward(ctx, *x, ends, ctx.saved(70, 1), out, *[torch.empty_like(y) for y in x])
    with pytest.raises(TypeError):
        ofrl.delta_backward(ctx, *x, ends, None, out, *[torch.empty_like(y) for y in x])
    state = torch.zeros(10, 2, 64, 64, device="cuda")
    with pytest.raises(ofrl.OfrlError):       # more tokens than states
        ofrl.delta_step(ctx, *x, state, out)
    more = _dev(np.zeros((71, 1, 64)))
    with pytest.raises(ofrl.OfrlError):       # more tokens than the context holds
        ofrl.delta_forward(ctx, more, more, _dev(np.zeros((71, 2, 64))), *[_dev(np.zeros((71, 2)))] * 2,
                           torch.tensor([71], dtype=torch.int32, device="cuda"), torch.empty(71, 2, 64, device="cuda"))
    # nothing to do is no error
    none = [y[:0] for y in x]
    ofrl.delta_forward(ctx, *none, ends[:0], out[:0])
    ofrl.delta_step(ctx, *none, state, out[:0])
    assert ctx.poll_status()["bad_index"] == 0
    ctx.close()
    for shape in ((1, 1, 0, 8), (2, 3, 64, 64), (0, 1, 64, 64)):
        with pytest.raises(ofrl.OfrlError, match="EINVAL"):
            ofrl.DeltaRule(*shape, "fp32")
    for shape in ((1, 1, 136, 64), (1, 1, 64, 136), (1, 1, 12, 64), (1, 1, 64, 4)):
        with pytest.raises(ofrl.OfrlError, match="EUNSUPPORTED"):
            ofrl.DeltaRule(*shape, "fp32")
