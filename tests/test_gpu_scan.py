"""GPU parity of the selective scan (forward, gradients, one token) against the fp64 recurrence."""
import numpy as np
import pytest
import torch

from _block import DT, ROUNDED, SCAN, SUM, check, dev, ends_of, host, junk, scan_inputs, strided
from _gpu import need_gpu
from oracle import block

pytestmark = pytest.mark.gpu

LENGTHS = {"one": [1], "short": [1, 2, 3, 16, 17, 15], "empty": [0, 3, 0, 0, 1, 2, 0], "mixed": [70, 1, 1, 33, 2, 129, 64, 8],
           "long": [700], "ones": [1] * 77, "edges": [64, 64, 16, 48, 128, 1, 63]}
ALL = ("D", "z", "dt_bias")


def _run(d, lengths, dtype, parts=ALL, states=True, grads=True, slices=False, softplus=True, ctx=None, own_saved=None):
    import offline_rl_step_gb300 as ofrl
    t, c = d["x"].shape
    groups, n = d["B"].shape[1:]
    e = len(lengths)
    own = ctx is None
    if own:
        ctx = ofrl.SelectiveScan(c, n, groups, dtype, softplus, max_tokens=t, max_episodes=e)
    x, dt, B, C, dout, z = (dev(d[k], dtype) for k in ("x", "dt", "B", "C", "dout", "z"))
    new = lambda v: junk(*v.shape, dtype=dtype)  # noqa: E731
    out, gx, gdt, gB, gC, gz = (new(v) for v in (x, x, dt, B, C, z))
    rest = []
    if slices:
        (x, z, dt), _ = strided([x, z, dt])
        (B, C), _ = strided([B, C], 3)
        (out, gx, gz, gdt), w1 = strided([out, gx, gz, gdt])
        (gB, gC), w2 = strided([gB, gC], 3)
        rest = [w1[:, 4 * c:], w2[:, 2 * groups * n:]]
    A = dev(d["A"])
    more = {k: (dev(d[k]) if k != "z" else z) if k in parts else None for k in ALL}
    ends = torch.from_numpy(ends_of(lengths)).cuda()
    init, final = (dev(d["init"]), junk(e, c, n)) if states else (None, None)
    saved = (ctx.saved(t).fill_(0xFF) if own_saved is None else own_saved) if grads else None
    ofrl.scan_forward(ctx, x, dt, A, B, C, ends, out, init_state=init, final_state=final, saved=saved, **more)
    res = {"out": out, "final": final}
    if grads:
        gA, gD, gb = junk(c, n), junk(c) if "D" in parts else None, junk(c) if "dt_bias" in parts else None
        dfin, dinit = (dev(d["d_final"]), junk(e, c, n)) if states else (None, None)
        ofrl.scan_backward(ctx, x, dt, A, B, C, ends, saved, dout, gx, gdt, gA, gB, gC, dD=gD, ddt_bias=gb,
                           dz=gz if "z" in parts else None, init_state=init, d_final=dfin, d_init=dinit, **more)
        res.update(x=gx, dt=gdt, A=gA, B=gB, C=gC, D=gD, dt_bias=gb, z=gz if "z" in parts else None, init=dinit)
    torch.cuda.synchronize()
    assert all((r == 0).all() for r in rest)
    assert ctx.poll_status()["bad_index"] == 0
    if own:
        ctx.close()
    return {k: host(v) for k, v in res.items()}


def _check(d, lengths, dtype, got, parts=ALL, states=True, softplus=True):
    ends = ends_of(lengths)
    args = [d[k] for k in ("x", "dt", "A", "B", "C")]
    more = {k: d[k] if k in parts else None for k in ALL}
    more.update(softplus=softplus, init=d["init"] if states else None)
    out, final = block.scan_forward(*args, ends, **more)
    rounded = ROUNDED[dtype]
    check(got["out"], out, SCAN + rounded, "out")
    if states:
        check(got["final"], final, SCAN, "final")
    if "x" not in got:
        return
    g = block.scan_backward(*args, ends, d["dout"], d_final=d["d_final"] if states else None, **more)
    for k in ("x", "dt", "B", "C"):
        check(got[k], g[k], SCAN + rounded, "d" + k)
    check(got["A"], g["A"], SUM, "dA")
    for k in ("D", "dt_bias"):
        if k in parts:
            check(got[k], g[k], SUM, "d" + k)
    if "z" in parts:
        check(got["z"], g["z"], SCAN + rounded, "dz")
    if states:
        check(got["init"], g["init"], SCAN, "d_init")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("lengths", list(LENGTHS), ids=str)
def test_parity(dtype, lengths):
    need_gpu()
    ln = LENGTHS[lengths]
    for i, (c, n, groups, parts, states, slices) in enumerate((
            (8, 16, 1, ALL, True, False), (24, 12, 1, ("z",), True, True), (48, 16, 2, ("D", "dt_bias"), False, True))):
        d = scan_inputs(ln, c, n, groups, 10 + i, dtype)
        _check(d, ln, dtype, _run(d, ln, dtype, parts, states, slices=slices), parts, states)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [4, 8, 12, 16, 20, 32, 44, 64])
def test_state_sizes(dtype, n):
    need_gpu()
    ln = [90, 0, 37, 300]
    d = scan_inputs(ln, 40, n, 1, n, dtype)
    _check(d, ln, dtype, _run(d, ln, dtype))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("c,n", [(1024, 4), (1000, 8), (1024, 16), (512, 28), (256, 64)])
def test_wide_calls(dtype, c, n):
    """Enough channels and tokens for several channels a thread."""
    need_gpu()
    ln = [1300, 700, 560]
    d = scan_inputs(ln, c, n, 1, 3, dtype)
    _check(d, ln, dtype, _run(d, ln, dtype, slices=True))


def test_groups():
    need_gpu()
    ln = [50, 90]
    for c, groups in ((64, 8), (72, 3), (1040, 2)):
        d = scan_inputs(ln, c, 16, groups, groups, "fp32")
        _check(d, ln, "fp32", _run(d, ln, "fp32"))


def test_deltas_as_they_are():
    need_gpu()
    ln = [50, 1, 90]
    d = scan_inputs(ln, 24, 16, 1, 5, "fp32", softplus=False)
    parts = ("D", "z")
    _check(d, ln, "fp32", _run(d, ln, "fp32", parts, softplus=False), parts, softplus=False)


def test_gradients_against_differences():
    """The gradients predict how the loss changes along themselves: fp32 tokens, differences of the library's own
    outputs summed in fp64.  The loss is off by SCAN times its terms' norm, the difference by that over the step."""
    need_gpu()
    ln = [40, 25]
    d = scan_inputs(ln, 16, 8, 1, 8, "fp32")
    g = _run(d, ln, "fp32")
    for k, eps in (("x", 0.05), ("dt", 0.02), ("B", 0.05), ("C", 0.05), ("z", 0.05), ("A", 0.02), ("D", 0.05),
                   ("dt_bias", 0.01)):
        v = g[k] / np.linalg.norm(g[k])
        losses = []
        for s in (-1, 1):
            moved = dict(d)
            moved[k] = np.float32(d[k] + s * eps * v)
            o = _run(moved, ln, "fp32", grads=False)
            losses.append((o["out"] * d["dout"]).sum() + (o["final"] * d["d_final"]).sum())
        want = np.linalg.norm(g[k])
        assert abs((losses[1] - losses[0]) / (2 * eps) - want) <= 0.01 * want, k


def test_edges_of_delta():
    """Deltas of zero leave the state, very large ones forget it; both exactly."""
    need_gpu()
    ln = [30]
    d = scan_inputs(ln, 8, 16, 1, 1, "fp32")
    d["dt"][10:20] = -np.inf      # softplus: 0
    d["dt"][20] = 3000.0
    d["x"][20] = 0.0
    got = _run(d, ln, "fp32")
    ends = ends_of(ln)
    out, final = block.scan_forward(*[d[k] for k in ("x", "dt", "A", "B", "C")], ends, d["D"], d["z"], d["dt_bias"], True,
                                    d["init"])
    check(got["out"], out, SCAN, "out")
    check(got["final"], final, SCAN, "final")
    state = _run(d, ln, "fp32", parts=("z", "dt_bias"))["out"]
    assert (state[20] == 0).all()      # everything before is forgotten


def test_small_steps_keep_their_bits():
    """dt far below zero: softplus is exp(dt), to fp32's relative precision."""
    need_gpu()
    ln = [60]
    d = scan_inputs(ln, 8, 8, 1, 2, "fp32")
    d["dt"] = np.float32(np.linspace(-30, -8, 60 * 8).reshape(60, 8))
    d["dt_bias"][:] = 0
    parts = ("z", "dt_bias")
    got = _run(d, ln, "fp32", parts, states=False)
    _check(d, ln, "fp32", got, parts, states=False)
    one = {k: (v[:1] if k in ("x", "dt", "B", "C", "z", "dout") else v) for k, v in d.items()}
    first = _run(one, [1], "fp32", ("z", "dt_bias"), states=False)["out"]
    want, _ = block.scan_forward(*[one[k] for k in ("x", "dt", "A", "B", "C")], [1], None, one["z"], one["dt_bias"])
    np.testing.assert_allclose(first, want, rtol=2e-5)


def test_steps_of_zero_keep_the_state():
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    t, c, n = 700, 16, 16
    d = scan_inputs([t], c, n, 1, 3, "fp32")
    d["dt"][:] = 0
    got = _run(d, [t], "fp32", parts=(), softplus=False)
    assert np.array_equal(got["final"], host(dev(d["init"])))
    assert not got["x"].any()
    ctx = ofrl.SelectiveScan(c, n, 1, "fp32", False, 0, 0, backward=False)
    x, dt, A, B, C = (dev(d[k][:1] if k != "A" else d[k]) for k in ("x", "dt", "A", "B", "C"))
    state = dev(d["init"])
    was = state.clone()
    for _ in range(10):
        ofrl.scan_step(ctx, x, dt, A, B, C, state, torch.empty_like(x))
    assert torch.equal(state, was)


def test_slow_states():
    """A state that remembers M = 120 tokens multiplies the mean error of a decay, 1.3e-8 at most, by M: 1.6e-6.  The
    roundings of the decays, 3e-8 each, and of the sums, at most 2^-24, are independent and add sqrt(M / 2) times
    themselves each: 2.3e-7 and 4.6e-7."""
    need_gpu()
    t, c, n = 3000, 64, 16
    d = scan_inputs([t], c, n, 1, 4, "fp32")
    rng = np.random.default_rng(5)
    d["dt"] = (rng.uniform(2.0 ** -7, 2.0 ** -6, (t, c)) * np.log(2)).astype(np.float32)
    d["x"], d["A"], d["B"] = np.ones_like(d["x"]), -np.ones_like(d["A"]), np.ones_like(d["B"])
    got = _run(d, [t], "fp32", parts=(), states=False, grads=False, softplus=False)
    want, _ = block.scan_forward(*(d[k] for k in ("x", "dt", "A", "B", "C")), ends_of([t]), softplus=False)
    assert np.linalg.norm(got["out"] - want) <= 2.3e-6 * np.linalg.norm(want)


def test_states_that_grow():
    """A above zero: nothing is clamped."""
    need_gpu()
    ln = [200, 30]
    d = scan_inputs(ln, 16, 16, 1, 4, "fp32")
    d["A"] = -0.05 * d["A"]
    got = _run(d, ln, "fp32")
    # a state here remembers all of its 200 tokens
    ends = ends_of(ln)
    out, final = block.scan_forward(*[d[k] for k in ("x", "dt", "A", "B", "C")], ends, d["D"], d["z"], d["dt_bias"], True,
                                    d["init"])
    check(got["out"], out, 200 * 2.0 ** -21, "out")
    check(got["final"], final, 200 * 2.0 ** -21, "final")


def test_tokens_behind_the_last_episode_stay():
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    lengths = [100, 60, 0]
    d = scan_inputs([200], 16, 16, 1, 0, "fp32")
    ctx = ofrl.SelectiveScan(16, 16, 1, "fp32", True, 200, 3)
    ends = torch.from_numpy(ends_of(lengths)).cuda()
    x, dt, B, C, z, dout = (dev(d[k]) for k in ("x", "dt", "B", "C", "z", "dout"))
    for v in (x, dt, B, C, z, dout):
        v[160:] = float("nan")
    out, gx, gdt, gB, gC, gz = (torch.full_like(v, 7.0) for v in (x, x, dt, B, C, z))
    gA, saved = junk(16, 16), ctx.saved(200).fill_(0xFF)
    ofrl.scan_forward(ctx, x, dt, dev(d["A"]), B, C, ends, out, z=z, saved=saved)
    ofrl.scan_backward(ctx, x, dt, dev(d["A"]), B, C, ends, saved, dout, gx, gdt, gA, gB, gC, z=z, dz=gz)
    for v in (out, gx, gdt, gB, gC, gz):
        assert (v[160:] == 7).all() and not (v[:160] == 7).any()
    cut = {k: v[:160] if k in ("x", "dt", "B", "C", "z", "dout") else v for k, v in d.items()}
    got = dict(out=out[:160], x=gx[:160], dt=gdt[:160], B=gB[:160], C=gC[:160], z=gz[:160], A=gA)
    _check(cut, lengths, "fp32", {k: host(v) for k, v in got.items()}, ("z",), states=False)


def test_no_tokens():
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    for n in (0, 3):
        ctx = ofrl.SelectiveScan(16, 8, 1, "bf16", True, 0, n)
        x = torch.empty(0, 16, device="cuda", dtype=DT["bf16"])
        B = torch.empty(0, 1, 8, device="cuda", dtype=DT["bf16"])
        A, gA, gD = -torch.ones(16, 8, device="cuda"), junk(16, 8), junk(16)
        ends = torch.zeros(n, dtype=torch.int32, device="cuda")
        init, final, dinit = torch.randn(n, 16, 8, device="cuda"), junk(n, 16, 8), junk(n, 16, 8)
        ofrl.scan_forward(ctx, x, x, A, B, B, ends, x, init_state=init, final_state=final, saved=ctx.saved(0))
        ofrl.scan_backward(ctx, x, x, A, B, B, ends, ctx.saved(0), x, x, x, gA, B, B, dD=gD, init_state=init, d_final=init,
                           d_init=dinit)
        assert torch.equal(final, init) and torch.equal(dinit, init)
        assert (gA == 0).all() and (gD == 0).all()


def test_bad_ends_are_counted():
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    t, c, n = 300, 16, 16
    d = scan_inputs([t], c, n, 1, 0, "fp32")
    ctx = ofrl.SelectiveScan(c, n, 1, "fp32", True, t, 4)
    x, dt, A, B, C = (dev(d[k]) for k in ("x", "dt", "A", "B", "C"))
    guard = torch.full((3, t, c), 5.0, device="cuda")
    states = torch.full((3, 4, c, n), 5.0, device="cuda")
    init = torch.zeros(4, c, n, device="cuda")
    for ends, bad in (([150, 40, 170, 300], 1), ([-3, 301, 20, 2 ** 30], 4), ([10, 20, 30, 2 ** 31 - 1], 1),
                      ([300, 200, 100, 0], 3), ([10, 20, 30, 300], 0)):
        e = torch.tensor(ends, dtype=torch.int32, device="cuda")
        saved = ctx.saved(t)
        ofrl.scan_forward(ctx, x, dt, A, B, C, e, guard[1], init_state=init, final_state=states[1], saved=saved)
        ofrl.scan_backward(ctx, x, dt, A, B, C, e, saved, x, guard[1], torch.empty_like(x), torch.empty_like(A),
                           torch.empty_like(B), torch.empty_like(C), init_state=init, d_final=init, d_init=states[1])
        assert ctx.poll_status()["bad_index"] == bad, ends
    for v in (guard, states):
        assert (v[0] == 5).all() and (v[2] == 5).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("what", ["x", "dt", "z", "B", "C"])
def test_non_finite_inputs_stay(bad, what):
    """They reach no earlier token, no other episode, no other channel (B and C: no other group)."""
    need_gpu()
    lengths = [100, 150, 90]
    d = scan_inputs(lengths, 32, 12, 2, 7, "fp32")
    clean = _run(d, lengths, "fp32")
    at = 160
    d[what][(at, 3) if what in ("x", "dt", "z") else (at, 1, 5)] = bad
    got = _run(d, lengths, "fp32")
    free = np.ones((340, 32), bool)      # what must not change
    if what in ("x", "dt", "z"):
        free[at:250, 3] = False
    else:
        free[at:250, 16:] = False
    assert (got["out"][free] == clean["out"][free]).all()
    assert (got["final"][[0, 2]] == clean["final"][[0, 2]]).all()
    others = [0, 1, 2] + list(range(4, 32)) if what in ("x", "dt", "z") else list(range(16))
    assert (got["final"][1][others] == clean["final"][1][others]).all()
    rows = np.r_[0:100, 250:340]
    for k in ("x", "dt", "z", "B", "C"):
        assert (got[k][rows] == clean[k][rows]).all(), k
    assert (got["init"][[0, 2]] == clean["init"][[0, 2]]).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("c,n,groups", [(8, 4, 1), (24, 16, 1), (144, 12, 2), (40, 64, 1), (264, 32, 1)])
def test_step_is_reading_one_token_at_a_time(dtype, c, n, groups):
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    envs, length = 5, 7
    lengths = [length] * envs
    d = scan_inputs(lengths, c, n, groups, 9, dtype)
    ctx = ofrl.SelectiveScan(c, n, groups, dtype, True, 0, 0, backward=False)
    v = {k: dev(d[k], dtype).view(envs, length, *d[k].shape[1:]) for k in ("x", "dt", "B", "C", "z")}
    A, D, b = dev(d["A"]), dev(d["D"]), dev(d["dt_bias"])
    state, other, outs = dev(d["init"]), junk(envs, c, n), []
    for i in range(length):
        out = junk(envs, c, dtype=dtype)
        args = (v["x"][:, i], v["dt"][:, i], A, v["B"][:, i], v["C"][:, i], state, out)
        if i % 2:
            ofrl.scan_step(ctx, *args, D=D, z=v["z"][:, i], dt_bias=b)
        else:
            ofrl.scan_step(ctx, *args, D=D, z=v["z"][:, i], dt_bias=b, new_state=other)
            state, other = other, state
        outs.append(out)
    _check(d, lengths, dtype, {"out": host(torch.stack(outs, 1).view(envs * length, c)), "final": host(state)})


def test_step_slots():
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    c, n, slots = 24, 16, 6
    d = scan_inputs([3], c, n, 1, 2, "fp32")
    ctx = ofrl.SelectiveScan(c, n, 1, "fp32", True, 0, 0, backward=False)
    args = [dev(d[k]) for k in ("x", "dt", "A", "B", "C")]
    state = torch.randn(slots, c, n, device="cuda")
    before, out = state.clone(), junk(3, c)
    ofrl.scan_step(ctx, *args, state, out, slots=torch.tensor([4, 6, 0], dtype=torch.int32, device="cuda"))
    assert ctx.poll_status()["bad_index"] == 1
    assert (out[1] == 0).all()
    for i, s in ((0, 4), (2, 0)):
        row = {k: d[k][i:i + 1] if k != "A" else d[k] for k in ("x", "dt", "A", "B", "C")}
        want, final = block.scan_forward(*row.values(), [1], init=host(before[s])[None])
        check(host(out[i]), want[0], SCAN, "out")
        check(host(state[s]), final[0], SCAN, "state")
    for s in (1, 2, 3, 5):
        assert torch.equal(state[s], before[s])


def test_streams_graphs_and_repeats():
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    lengths, c, n = [100, 0, 333, 500], 72, 16
    d = scan_inputs(lengths, c, n, 1, 6, "bf16")
    want = _run(d, lengths, "bf16")
    again = _run(d, lengths, "bf16")
    assert all((want[k] == again[k]).all() for k in want)
    t, e = 933, 4
    ctx = ofrl.SelectiveScan(c, n, 1, "bf16", True, t, e)
    x, dt, B, C, z, dout = (dev(d[k], "bf16") for k in ("x", "dt", "B", "C", "z", "dout"))
    A, D, b, init, dfin = (dev(d[k]) for k in ("A", "D", "dt_bias", "init", "d_final"))
    ends, saved = torch.from_numpy(ends_of(lengths)).cuda(), ctx.saved(t)
    o = {k: torch.empty_like(v) for k, v in dict(out=x, x=x, dt=dt, B=B, C=C, z=z, A=A, D=D, dt_bias=b, final=init,
                                                 init=init).items()}

    def both():
        ofrl.scan_forward(ctx, x, dt, A, B, C, ends, o["out"], D=D, z=z, dt_bias=b, init_state=init, final_state=o["final"],
                          saved=saved)
        ofrl.scan_backward(ctx, x, dt, A, B, C, ends, saved, dout, o["x"], o["dt"], o["A"], o["B"], o["C"], D=D, z=z,
                           dt_bias=b, dD=o["D"], dz=o["z"], ddt_bias=o["dt_bias"], init_state=init, d_final=dfin,
                           d_init=o["init"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.synchronize()
    assert all((host(o[k]) == want[k]).all() for k in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for _ in range(2):
        for v in o.values():
            v.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all((host(o[k]) == want[k]).all() for k in want)


def test_a_workspace_serves_smaller_calls():
    """One context, calls of every size up to what it was made for."""
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    ctx = ofrl.SelectiveScan(64, 16, 1, "fp32", True, 3000, 8)
    saved = ctx.saved(3000)
    for ln in ([3000], [1], [17, 64], [1000, 0, 500]):
        d = scan_inputs(ln, 64, 16, 1, 1, "fp32")
        _check(d, ln, "fp32", _run(d, ln, "fp32", ctx=ctx, own_saved=saved))


def test_states_carry_a_split_trajectory():
    """Reading in two calls, the state handed on, is reading at once."""
    need_gpu()
    ln = [500]
    d = scan_inputs(ln, 24, 16, 1, 3, "fp32")
    whole = _run(d, ln, "fp32", grads=False)
    rows = ("x", "dt", "B", "C", "z", "dout")
    a = _run({k: v[:213] if k in rows else v for k, v in d.items()}, [213], "fp32", grads=False)
    second = {k: v[213:] if k in rows else v for k, v in d.items()}
    second["init"] = np.float32(a["final"])
    b = _run(second, [287], "fp32", grads=False)
    check(np.concatenate([a["out"], b["out"]]), whole["out"], SCAN, "out")
    check(b["final"], whole["final"], SCAN, "final")


def test_refusals():
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    t, c, n = 100, 16, 16
    ctx = ofrl.SelectiveScan(c, n, 1, "bf16", True, t, 4)
    bf = DT["bf16"]
    x = torch.zeros(t, c, device="cuda", dtype=bf)
    B = torch.zeros(t, 1, n, device="cuda", dtype=bf)
    A = -torch.ones(c, n, device="cuda")
    ends = torch.tensor([t], dtype=torch.int32, device="cuda")
    out, wide = torch.zeros_like(x), torch.zeros(t, 64, device="cuda", dtype=bf)

    def refused(error, *a, **k):
        with pytest.raises(error):
            ofrl.scan_forward(ctx, *a, **k)

    refused(TypeError, x.float(), x, A, B, B, ends, out)
    refused(TypeError, x, x, A.bfloat16(), B, B, ends, out)
    refused(TypeError, x, x, None, B, B, ends, out)
    refused(ValueError, x, x, A, B[:, :, :8], B, ends, out)
    refused(ValueError, x, x, A.T[:8], B, B, ends, out)
    refused(ValueError, x, x[:50], A, B, B, ends, out)
    refused(ValueError, x, x, A, B, B, ends, out, D=torch.zeros(8, device="cuda"))
    refused(ofrl.OfrlError, wide[:, 4:20], x, A, B, B, ends, out)
    refused(ofrl.OfrlError, x, x, A, B, B, ends, out, z=wide[:, 4:20])
    refused(ofrl.OfrlError, x[:1].expand(t, c), x, A, B, B, ends, out)
    refused(ofrl.OfrlError, x, x, A, B, B, ends[:0], out)
    refused(ofrl.OfrlError, x, x, A, B, B, torch.full((5,), t, dtype=torch.int32, device="cuda"), out)
    refused(ValueError, x, x, A, B, B, ends, out, saved=torch.empty(8, device="cuda", dtype=torch.uint8))
    refused(TypeError, x, x, A, B, B, ends, out, init_state=torch.zeros(1, c, n, device="cuda", dtype=bf))
    off = torch.zeros(c * n + 1, device="cuda")[1:].view(c, n)      # off 16 bytes
    refused(ofrl.OfrlError, x, x, off, B, B, ends, out)
    more = torch.zeros(t + 1, c, device="cuda", dtype=bf)
    refused(ofrl.OfrlError, more, more, A, torch.zeros(t + 1, 1, n, device="cuda", dtype=bf),
            torch.zeros(t + 1, 1, n, device="cuda", dtype=bf), ends, torch.zeros_like(more))
    saved, gA = ctx.saved(t), torch.zeros_like(A)

    def back(error, *a, **k):
        with pytest.raises(error):
            ofrl.scan_backward(ctx, x, x, A, B, B, ends, *a, **k)

    back(TypeError, None, x, out, out, gA, B, B)
    back(TypeError, saved, x, out, out, None, B, B)
    back(ofrl.OfrlError, saved, x, out, out, gA, B, B, z=x)            # a gate without its gradient
    back(ofrl.OfrlError, saved, x, out, out, gA, B, B, dz=out)         # and the other way round
    forward_only = ofrl.SelectiveScan(c, n, 1, "bf16", True, t, 4, backward=False)
    with pytest.raises(ofrl.OfrlError):
        ofrl.scan_backward(forward_only, x, x, A, B, B, ends, saved, x, out, out, gA, B, B)
    with pytest.raises(ofrl.OfrlError):
        ofrl.scan_step(ctx, x[:4], x[:4], A, B[:4], B[:4], torch.zeros(3, c, n, device="cuda"), out[:4])
    ctx.close()
    with pytest.raises(ValueError, match="closed"):
        ofrl.scan_forward(ctx, x, x, A, B, B, ends, out)
