"""State space blocks: calls that are refused for where their buffers are, and first calls under capture."""
import os
import subprocess
import sys

import pytest
import torch

from _block import dev, ends_of, junk, scan_inputs, conv_inputs
from _gpu import need_gpu

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_states_that_overlap_are_refused():
    """Parts of one episode run at the same time: its final state may be written before its initial one is read."""
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    ln, c, n = [40, 30], 16, 16
    d = scan_inputs(ln, c, n, 1, 0, "fp32")
    ctx = ofrl.SelectiveScan(c, n, 1, "fp32", True, 70, 2)
    x, dt, A, B, C, dout = (dev(d[k]) for k in ("x", "dt", "A", "B", "C", "dout"))
    ends = torch.from_numpy(ends_of(ln)).cuda()
    both = torch.zeros(3, c, n, device="cuda")
    out, saved = torch.empty_like(x), ctx.saved(70)
    for a, b in ((both[:2], both[:2]), (both[:2], both[1:]), (both[1:], both[:2])):
        with pytest.raises(ofrl.OfrlError):
            ofrl.scan_forward(ctx, x, dt, A, B, C, ends, out, init_state=a, final_state=b)
        for k in (dict(d_final=a, d_init=b), dict(init_state=a, d_init=b)):
            with pytest.raises(ofrl.OfrlError):
                ofrl.scan_backward(ctx, x, dt, A, B, C, ends, saved, dout, out, torch.empty_like(x), torch.empty_like(A),
                                   torch.empty_like(B), torch.empty_like(C), **k)
    apart = torch.zeros(4, c, n, device="cuda")
    ofrl.scan_forward(ctx, x, dt, A, B, C, ends, out, init_state=apart[:2], final_state=apart[2:], saved=saved)
    # a gradient of the final states and the initial ones may share a buffer: both are only read
    ofrl.scan_backward(ctx, x, dt, A, B, C, ends, saved, dout, torch.empty_like(x), torch.empty_like(x), torch.empty_like(A),
                       torch.empty_like(B), torch.empty_like(C), init_state=apart[:2], d_final=apart[:2], d_init=both[:2])

    d = conv_inputs(ln, c, 4, 0, "fp32")
    ctx = ofrl.CausalConv(c, 4, "silu", "fp32", 70, 2)
    x, w = dev(d["x"]), dev(d["w"])
    both = torch.zeros(3, c, 3, device="cuda")
    for a, b in ((both[:2], both[:2]), (both[:2], both[1:])):
        with pytest.raises(ofrl.OfrlError):
            ofrl.conv_forward(ctx, x, w, ends, out, init_state=a, final_state=b)
        with pytest.raises(ofrl.OfrlError):
            ofrl.conv_backward(ctx, x, w, ends, x, out, torch.empty_like(w), d_final=a, d_init=b)


def test_tensors_of_another_device_are_refused():
    """Seen from a workspace that says it is elsewhere: nothing is launched."""
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    x, w = torch.zeros(10, 16, device="cuda"), torch.zeros(16, 4, device="cuda")
    ends, one = torch.tensor([10], dtype=torch.int32, device="cuda"), torch.ones(16, device="cuda")
    B, A, out = torch.zeros(10, 1, 8, device="cuda"), -torch.ones(16, 8, device="cuda"), torch.full((10, 16), 3.0, device="cuda")
    conv, scan, norm = (ofrl.CausalConv(16, 4, "silu", "fp32", 10, 1), ofrl.SelectiveScan(16, 8, 1, "fp32", True, 10, 1),
                        ofrl.BlockNorm(16, 1, "fp32"))
    saved, conv_state, scan_state = scan.saved(10), torch.zeros(10, 16, 3, device="cuda"), torch.zeros(10, 16, 8, device="cuda")
    calls = (lambda: ofrl.conv_forward(conv, x, w, ends, out), lambda: ofrl.conv_backward(conv, x, w, ends, x, out, w.clone()),
             lambda: ofrl.conv_step(conv, x, w, conv_state, out), lambda: ofrl.scan_forward(scan, x, x, A, B, B, ends, out),
             lambda: ofrl.scan_backward(scan, x, x, A, B, B, ends, saved, x, out, out, A, B, B),
             lambda: ofrl.scan_step(scan, x, x, A, B, B, scan_state, out), lambda: ofrl.gated_norm(norm, x, x, one, out),
             lambda: ofrl.gated_norm_backward(norm, x, x, one, x, out, out, one.clone()),
             lambda: ofrl.residual_norm(norm, x, x, one, out, out),
             lambda: ofrl.residual_norm_backward(norm, x, x, one, x, out, out, one.clone()))
    for ctx in (conv, scan, norm):
        ctx.device += 1
    for call in calls:
        with pytest.raises(ValueError, match="must be on cuda:1"):
            call()
    for ctx in (conv, scan, norm):
        ctx.device -= 1
    assert (out == 3).all()


FIRST = r"""
import sys
sys.path.insert(0, sys.argv[1])
import torch
import offline_rl_step_gb300 as ofrl
t, c, n = 300, 64, 16
x = torch.randn(t, c, device="cuda")
B, A = torch.randn(t, 1, n, device="cuda"), -torch.rand(c, n, device="cuda") - 0.5
w, one, ends = torch.randn(c, 4, device="cuda"), torch.ones(c, device="cuda"), torch.tensor([100, 300], dtype=torch.int32, device="cuda")
conv, scan, norm = (ofrl.CausalConv(c, 4, "silu", "fp32", t, 2), ofrl.SelectiveScan(c, n, 1, "fp32", True, t, 2),
                    ofrl.BlockNorm(c, 1, "fp32"))
saved, o = scan.saved(t), [torch.empty_like(x) for _ in range(9)]
dw, dA, dB, dC, dn = torch.empty_like(w), torch.empty_like(A), torch.empty_like(B), torch.empty_like(B), torch.empty_like(one)

def block():
    ofrl.conv_forward(conv, x, w, ends, o[0])
    ofrl.scan_forward(scan, o[0], x, A, B, B, ends, o[1], z=x, saved=saved)
    ofrl.gated_norm(norm, o[1], x, one, o[2])
    ofrl.residual_norm(norm, o[2], x, one, o[3], o[4])
    ofrl.residual_norm_backward(norm, o[2], x, one, x, o[5], o[6], dn)
    ofrl.gated_norm_backward(norm, o[1], x, one, o[5], o[6], o[7], dn)
    ofrl.scan_backward(scan, o[0], x, A, B, B, ends, saved, o[6], o[5], o[7], dA, dB, dC, z=x, dz=o[8])
    ofrl.conv_backward(conv, x, w, ends, o[5], o[6], dw)

torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    block()
g.replay()
torch.cuda.synchronize()
got = [v.clone() for v in o + [dw, dA, dB, dC, dn]]
block()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, o + [dw, dA, dB, dC, dn]))
print("the same")
"""


def test_first_calls_may_be_captured():
    need_gpu()
    r = subprocess.run([sys.executable, "-c", FIRST, ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "the same" in r.stdout, r.stderr[-2000:]


def test_two_graphs_share_a_workspace():
    """Captured one after the other with one context, replayed in turn on one stream."""
    import offline_rl_step_gb300 as ofrl
    need_gpu()
    c, n = 48, 16
    ctx = ofrl.SelectiveScan(c, n, 1, "bf16", True, 1000, 4)
    graphs, outs, wants = [], [], []
    for ln in ([600, 400], [33, 0, 200]):
        t = sum(ln)
        d = scan_inputs(ln, c, n, 1, t, "bf16")
        x, dt, B, C = (dev(d[k], "bf16") for k in ("x", "dt", "B", "C"))
        A, ends, out = dev(d["A"]), torch.from_numpy(ends_of(ln)).cuda(), junk(t, c, dtype="bf16")
        ofrl.scan_forward(ctx, x, dt, A, B, C, ends, out)
        torch.cuda.synchronize()
        wants.append(out.clone())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ofrl.scan_forward(ctx, x, dt, A, B, C, ends, out)
        graphs.append((g, x, dt, A, B, C, ends))
        outs.append(out)
    for _ in range(3):
        for g, out, want in zip(graphs, outs, wants):
            out.fill_(float("nan"))
            g[0].replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
