"""GPU parity of the gated norm and the residual norm with their gradients against fp64."""
import numpy as np
import pytest
import torch

from _block import DT, ROUND, ROUNDED, ROW, SUM, check, dev, host, junk, strided
from _gpu import need_gpu
from oracle import block

pytestmark = pytest.mark.gpu

# channels, groups: one vector, odd counts, sub-warps, a warp, whole CTAs of each size
SHAPES = [(8, 1), (24, 1), (64, 2), (200, 1), (264, 3), (512, 1), (520, 1), (1024, 1), (1000, 5), (2056, 1), (4096, 1), (8192, 1),
          (4112, 2)]


def _inputs(rows, c, seed, dtype, residual="fp32"):
    r, rnd = np.random.default_rng(seed), ROUND[dtype]
    n = lambda *s: r.standard_normal(s)  # noqa: E731
    return dict(x=rnd(n(rows, c)), z=rnd(n(rows, c)), w=np.float32(1 + 0.3 * n(c)), dout=rnd(n(rows, c)),
                residual=ROUND[residual](2 * n(rows, c)), scale=np.float32(n(c)), dres=ROUND[residual](n(rows, c)))


def _gated(d, groups, dtype, gate_first, eps=1e-5, slices=False):
    import offline_rl_step_gb300 as ofrl
    rows, c = d["x"].shape
    ctx = ofrl.BlockNorm(c, groups, dtype)
    x, z, g = (dev(d[k], dtype) for k in ("x", "z", "dout"))
    out, dx, dz, dw = junk(rows, c, dtype=dtype), junk(rows, c, dtype=dtype), junk(rows, c, dtype=dtype), junk(c)
    if slices:
        (x, z, g), _ = strided([x, z, g])
        (out, dx, dz), wide = strided([out, dx, dz])
    w = dev(d["w"])
    ofrl.gated_norm(ctx, x, z, w, out, eps=eps, gate_first=gate_first)
    ofrl.gated_norm_backward(ctx, x, z, w, g, dx, dz, dw, eps=eps, gate_first=gate_first)
    torch.cuda.synchronize()
    if slices:
        assert (wide[:, 3 * c:] == 0).all()
    ctx.close()
    return [host(v) for v in (out, dx, dz, dw)]


def _residual(d, groups, dtype, residual, scaled, dres=True, eps=1e-5, slices=False):
    import offline_rl_step_gb300 as ofrl
    rows, c = d["x"].shape
    ctx = ofrl.BlockNorm(c, groups, dtype, residual)
    x, g = dev(d["x"], dtype), dev(d["dout"], dtype)
    r, dr = dev(d["residual"], residual), dev(d["dres"], residual) if dres else None
    out, dx = junk(rows, c, dtype=dtype), junk(rows, c, dtype=dtype)
    res, gr = junk(rows, c, dtype=residual), junk(rows, c, dtype=residual)
    if slices:
        (x, g), _ = strided([x, g])
        (out, dx), w1 = strided([out, dx])
        (res, gr), w2 = strided([res, gr])
    w, s = dev(d["w"]), dev(d["scale"]) if scaled else None
    dw, ds = junk(c), junk(c) if scaled else None
    ofrl.residual_norm(ctx, x, r, w, res, out, scale=s, eps=eps)
    ofrl.residual_norm_backward(ctx, x, r, w, g, dx, gr, dw, scale=s, dscale=ds, d_residual_out=dr, eps=eps)
    torch.cuda.synchronize()
    if slices:
        assert (w1[:, 2 * c:] == 0).all() and (w2[:, 2 * c:] == 0).all()
    ctx.close()
    return [host(v) for v in (res, out, dx, gr, dw, ds)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("c,groups", SHAPES)
@pytest.mark.parametrize("gate_first", [False, True])
def test_gated(dtype, c, groups, gate_first):
    need_gpu()
    for rows, slices in ((1, False), (7, True), (301, True)):
        d = _inputs(rows, c, rows + c, dtype)
        got = _gated(d, groups, dtype, gate_first, slices=slices)
        bound = ROW + ROUNDED[dtype]
        check(got[0], block.gated_norm(d["x"], d["z"], d["w"], groups, gate_first=gate_first), bound, "out")
        want = block.gated_norm_backward(d["x"], d["z"], d["w"], d["dout"], groups, gate_first=gate_first)
        check(got[1], want[0], bound, "dx")
        check(got[2], want[1], bound, "dz")
        check(got[3], want[2], SUM, "dw")


@pytest.mark.parametrize("dtype,residual", [("fp32", "fp32"), ("bf16", "bf16"), ("bf16", "fp32")])
@pytest.mark.parametrize("c,groups", SHAPES)
def test_residual(dtype, residual, c, groups):
    need_gpu()
    for rows, scaled, dres, slices in ((1, True, True, False), (7, False, True, True), (301, True, False, True)):
        d = _inputs(rows, c, rows + c, dtype, residual)
        got = _residual(d, groups, dtype, residual, scaled, dres, slices=slices)
        s = d["scale"] if scaled else None
        h, out = block.residual_norm(d["x"], d["residual"], d["w"], s, groups)
        check(got[0], h, ROW + ROUNDED[residual], "residual_out")
        check(got[1], out, ROW + ROUNDED[dtype], "out")
        want = block.residual_norm_backward(d["x"], d["residual"], d["w"], d["dout"], s, d["dres"] if dres else None, groups)
        check(got[2], want[0], ROW + ROUNDED[dtype], "dx")
        check(got[3], want[1], ROW + ROUNDED[residual], "dresidual")
        check(got[4], want[2], SUM, "dw")
        if scaled:
            check(got[5], want[3], SUM, "dscale")


def test_many_rows():
    """More rows than the grid has seats: every thread takes several."""
    need_gpu()
    for c, groups, rows in ((16, 1, 200001), (72, 3, 30011), (1032, 1, 9001)):
        d = _inputs(rows, c, 1, "bf16")
        got = _gated(d, groups, "bf16", True)
        check(got[0], block.gated_norm(d["x"], d["z"], d["w"], groups, gate_first=True), ROW + ROUNDED["bf16"], "out")
        # a column sums 200 thousand terms of either sign: against the norm of all columns
        check(got[3], block.gated_norm_backward(d["x"], d["z"], d["w"], d["dout"], groups, gate_first=True)[2], SUM, "dw")


def test_no_rows():
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    ctx = ofrl.BlockNorm(64, 1, "bf16")
    x, w = torch.empty(0, 64, device="cuda", dtype=DT["bf16"]), torch.ones(64, device="cuda")
    dw, ds = junk(64), junk(64)
    ofrl.gated_norm(ctx, x, x, w, x)
    ofrl.gated_norm_backward(ctx, x, x, w, x, x, x, dw)
    assert (dw == 0).all()
    dw.fill_(float("nan"))
    ofrl.residual_norm(ctx, x, x, w, x, x)
    ofrl.residual_norm_backward(ctx, x, x, w, x, x, x, dw, scale=w, dscale=ds)
    assert (dw == 0).all() and (ds == 0).all()


def test_rows_of_zeros_and_of_large_numbers():
    need_gpu()
    for c in (64, 2056):
        d = _inputs(6, c, 3, "fp32")
        d["x"][0], d["residual"][0], d["z"][1] = 0, 0, 0
        d["x"][2] *= 1e15
        d["x"][3] *= 1e-15
        d["z"][4] = -200.0      # the gate is zero
        for first in (False, True):
            got = _gated(d, 1, "fp32", first)
            assert all(np.isfinite(v).all() for v in got)
            want = block.gated_norm(d["x"], d["z"], d["w"], gate_first=first)
            np.testing.assert_allclose(got[0], want, rtol=1e-5, atol=1e-12)
        got = _residual(d, 1, "fp32", "fp32", False)
        assert all(np.isfinite(v).all() for v in got if v is not None)
        np.testing.assert_allclose(got[1], block.residual_norm(d["x"], d["residual"], d["w"])[1], rtol=1e-5, atol=1e-9)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("c,groups", [(128, 2), (4112, 2)])
def test_non_finite_inputs_stay_in_their_row_and_group(bad, c, groups):
    need_gpu()
    d = _inputs(9, c, 5, "fp32")
    clean = _gated(d, groups, "fp32", False), _residual(d, groups, "fp32", "fp32", True)
    d["x"][4, 3] = bad
    got = _gated(d, groups, "fp32", False), _residual(d, groups, "fp32", "fp32", True)
    free = np.ones((9, c), bool)
    free[4, :c // groups] = False
    for i in range(3):
        assert (got[0][i][free] == clean[0][i][free]).all()
    for i in range(4):
        assert (got[1][i][free] == clean[1][i][free]).all()
    half = slice(c // groups, None)
    assert (got[0][3][half] == clean[0][3][half]).all() and (got[1][4][half] == clean[1][4][half]).all()


def test_in_place():
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    for c in (72, 2056):
        d = _inputs(50, c, 8, "bf16", "bf16")
        want, want_r = _gated(d, 1, "bf16", False), _residual(d, 1, "bf16", "bf16", True)
        ctx = ofrl.BlockNorm(c, 1, "bf16")
        x, z, g, w, s = dev(d["x"], "bf16"), dev(d["z"], "bf16"), dev(d["dout"], "bf16"), dev(d["w"]), dev(d["scale"])
        y = x.clone()
        ofrl.gated_norm(ctx, y, z, w, y)
        assert (host(y) == want[0]).all()
        dx, dz, dw = g.clone(), z.clone(), junk(c)
        ofrl.gated_norm_backward(ctx, x, dz, w, dx, dx, dz, dw)
        assert (host(dx) == want[1]).all() and (host(dz) == want[2]).all() and (host(dw) == want[3]).all()
        y, r = x.clone(), dev(d["residual"], "bf16")
        ofrl.residual_norm(ctx, y, r, w, r, y, scale=s)
        assert (host(r) == want_r[0]).all() and (host(y) == want_r[1]).all()
        dx, dr, ds = g.clone(), dev(d["dres"], "bf16"), junk(c)
        ofrl.residual_norm_backward(ctx, x, dev(d["residual"], "bf16"), w, dx, dx, dr, dw, scale=s, dscale=ds,
                                    d_residual_out=dr)
        assert (host(dx) == want_r[2]).all() and (host(dr) == want_r[3]).all()
        assert (host(dw) == want_r[4]).all() and (host(ds) == want_r[5]).all()


def test_streams_graphs_and_repeats():
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    rows, c = 700, 520
    d = _inputs(rows, c, 2, "bf16")
    want = _gated(d, 1, "bf16", True)
    assert all((a == b).all() for a, b in zip(want, _gated(d, 1, "bf16", True)))
    ctx = ofrl.BlockNorm(c, 1, "bf16")
    x, z, g, w = (dev(d[k], "bf16") if k != "w" else dev(d[k]) for k in ("x", "z", "dout", "w"))
    o = [torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)]

    def both():
        ofrl.gated_norm(ctx, x, z, w, o[0], gate_first=True)
        ofrl.gated_norm_backward(ctx, x, z, w, g, *o[1:], gate_first=True)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.synchronize()
    assert all((host(a) == b).all() for a, b in zip(o, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for _ in range(2):
        for v in o:
            v.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all((host(a) == b).all() for a, b in zip(o, want))


def test_refusals():
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    ctx = ofrl.BlockNorm(64, 1, "bf16", "fp32")
    x, w = torch.zeros(10, 64, device="cuda", dtype=DT["bf16"]), torch.ones(64, device="cuda")
    r = torch.zeros(10, 64, device="cuda")
    wide = torch.zeros(10, 128, device="cuda", dtype=DT["bf16"])
    out = torch.zeros_like(x)
    for error, args, more in ((TypeError, (x.float(), x, w, out), {}), (TypeError, (x, x, None, out), {}),
                              (ValueError, (x, x[:5], w, out), {}), (ValueError, (x, x, w[:32], out), {}),
                              (ValueError, (wide[:, ::2], x, w, out), {}), (ofrl.OfrlError, (wide[:, 4:68], x, w, out), {}),
                              (ofrl.OfrlError, (x, x, w, out), dict(eps=0.0)),
                              (ofrl.OfrlError, (x, x, w, out), dict(eps=float("inf"))),
                              (ofrl.OfrlError, (x, x, torch.zeros(65, device="cuda")[1:], out), {})):
        with pytest.raises(error):
            ofrl.gated_norm(ctx, *args, **more)
    with pytest.raises(TypeError):
        ofrl.residual_norm(ctx, x, x, w, r, out)                          # the residual is fp32
    with pytest.raises(ofrl.OfrlError):
        ofrl.residual_norm_backward(ctx, x, r, w, x, out, r, torch.empty_like(w), scale=w)      # dscale is missing
    with pytest.raises(ofrl.OfrlError):
        ofrl.residual_norm_backward(ctx, x, r, w, x, out, r, torch.empty_like(w), dscale=torch.empty_like(w))
    forward_only = ofrl.BlockNorm(64, 1, "bf16", backward=False)
    with pytest.raises(ofrl.OfrlError):
        ofrl.gated_norm_backward(forward_only, x, x, w, x, out, out.clone(), torch.empty_like(w))
    with pytest.raises(ofrl.OfrlError):
        ofrl.BlockNorm(64, 1, "fp32", "bf16")
    ctx.close()
    with pytest.raises(ValueError, match="closed"):
        ofrl.gated_norm(ctx, x, x, w, out)
