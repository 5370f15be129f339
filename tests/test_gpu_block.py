"""A state space block as it is used: residual norm, convolution, scan and gated norm with plain projections between
them, trained over packed episodes and then acting one step at a time."""
import numpy as np
import pytest
import torch
import torch.nn.functional as F

from _block import check, ends_of, host
from _gpu import need_gpu

pytestmark = pytest.mark.gpu

DIM, INNER, N, RANK, WIDTH, EPS = 24, 48, 16, 8, 4, 1e-5


def _params(seed):
    g = torch.Generator().manual_seed(seed)
    new = lambda *s: (torch.randn(*s, generator=g) * s[0] ** -0.5).cuda()  # noqa: E731
    return dict(scale=1 + 0.1 * new(DIM), w_pre=1 + 0.1 * new(DIM), w_in=new(DIM, 2 * INNER), conv=new(INNER, WIDTH),
                conv_bias=0.1 * new(INNER), w_bc=new(INNER, RANK + 2 * N), w_dt=new(RANK, INNER), dt_bias=new(INNER) - 1,
                A=-torch.exp(new(INNER, N)), D=1 + 0.1 * new(INNER), w_post=1 + 0.1 * new(INNER), w_out=new(INNER, DIM))


class Block:
    """The library's block: forward keeps what backward takes."""

    def __init__(self, tokens, episodes):
        import offline_rl_step_gb300 as ofrl
        self.ofrl = ofrl
        self.pre = ofrl.BlockNorm(DIM, 1, "fp32")
        self.conv = ofrl.CausalConv(INNER, WIDTH, "silu", "fp32", tokens, episodes)
        self.scan = ofrl.SelectiveScan(INNER, N, 1, "fp32", True, tokens, episodes)
        self.post = ofrl.BlockNorm(INNER, 2, "fp32")
        self.saved = self.scan.saved(tokens)

    def forward(self, p, x, residual, ends):
        o, k = self.ofrl, {}
        k["h"], k["normed"] = torch.empty_like(x), torch.empty_like(x)
        o.residual_norm(self.pre, x, residual, p["w_pre"], k["h"], k["normed"], scale=p["scale"], eps=EPS)
        k["xz"] = k["normed"] @ p["w_in"]
        u, z = k["xz"].split(INNER, 1)
        k["u"], k["z"], k["c"] = u, z, torch.empty(x.shape[0], INNER, device="cuda")
        o.conv_forward(self.conv, u, p["conv"], ends, k["c"], bias=p["conv_bias"])
        k["low"] = k["c"] @ p["w_bc"]
        k["dt"] = k["low"][:, :RANK] @ p["w_dt"]
        k["B"], k["C"] = k["low"][:, RANK:RANK + N].unsqueeze(1), k["low"][:, RANK + N:].unsqueeze(1)
        k["y"], k["g"] = torch.empty_like(k["c"]), torch.empty_like(k["c"])
        o.scan_forward(self.scan, k["c"], k["dt"], p["A"], k["B"], k["C"], ends, k["y"], D=p["D"], dt_bias=p["dt_bias"],
                       saved=self.saved)
        o.gated_norm(self.post, k["y"], z, p["w_post"], k["g"], eps=EPS)
        k["x"], k["residual"] = x, residual
        return k["g"] @ p["w_out"], k["h"], k

    def backward(self, p, k, ends, dout, dh):
        o = self.ofrl
        g = {n: torch.empty_like(v) for n, v in p.items()}
        g["w_out"] = k["g"].T @ dout
        dg, dxz = dout @ p["w_out"].T, torch.empty_like(k["xz"])
        du, dz = dxz.split(INNER, 1)
        dy = torch.empty_like(dg)
        o.gated_norm_backward(self.post, k["y"], k["z"], p["w_post"], dg, dy, dz, g["w_post"], eps=EPS)
        dc, ddt, dlow = torch.empty_like(dy), torch.empty_like(dy), torch.empty_like(k["low"])
        dB, dC = dlow[:, RANK:RANK + N].unsqueeze(1), dlow[:, RANK + N:].unsqueeze(1)
        o.scan_backward(self.scan, k["c"], k["dt"], p["A"], k["B"], k["C"], ends, self.saved, dy, dc, ddt, g["A"], dB, dC,
                        D=p["D"], dt_bias=p["dt_bias"], dD=g["D"], ddt_bias=g["dt_bias"])
        g["w_dt"] = k["low"][:, :RANK].T @ ddt
        dlow[:, :RANK] = ddt @ p["w_dt"].T
        g["w_bc"] = k["c"].T @ dlow
        dc = dc + dlow @ p["w_bc"].T
        o.conv_backward(self.conv, k["u"], p["conv"], ends, dc, du, g["conv"], bias=p["conv_bias"], dbias=g["conv_bias"])
        g["w_in"] = k["normed"].T @ dxz
        dn = dxz @ p["w_in"].T
        dx, dr = torch.empty_like(dn), torch.empty_like(dn)
        o.residual_norm_backward(self.pre, k["x"], k["residual"], p["w_pre"], dn, dx, dr, g["w_pre"], scale=p["scale"],
                                 dscale=g["scale"], d_residual_out=dh, eps=EPS)
        return dx, dr, g

    def act(self, p, x, residual, conv_state, scan_state):
        """One token of every environment; the states move on in place."""
        o = self.ofrl
        h, n = torch.empty_like(x), torch.empty_like(x)
        o.residual_norm(self.pre, x, residual, p["w_pre"], h, n, scale=p["scale"], eps=EPS)
        u, z = (n @ p["w_in"]).split(INNER, 1)
        c = torch.empty(x.shape[0], INNER, device="cuda")
        o.conv_step(self.conv, u, p["conv"], conv_state, c, bias=p["conv_bias"])
        low = c @ p["w_bc"]
        y = torch.empty_like(c)
        o.scan_step(self.scan, c, low[:, :RANK] @ p["w_dt"], p["A"], low[:, RANK:RANK + N].unsqueeze(1),
                    low[:, RANK + N:].unsqueeze(1), scan_state, y, D=p["D"], dt_bias=p["dt_bias"])
        o.gated_norm(self.post, y, z, p["w_post"], y, eps=EPS)
        return y @ p["w_out"], h


def _plain(p, x, residual, lengths):
    """The block in fp64 with torch's own operators, one episode after the other."""
    h = residual + p["scale"] * x
    normed = F.rms_norm(h, (DIM,), eps=EPS) * p["w_pre"]
    u, z = (normed @ p["w_in"]).split(INNER, 1)
    ys, lo = [], 0
    for n in lengths:
        if n == 0:
            continue
        v = F.pad(u[lo:lo + n].T, (WIDTH - 1, 0))
        c = F.silu(F.conv1d(v[None], p["conv"][:, None], p["conv_bias"], groups=INNER)[0].T)
        low = c @ p["w_bc"]
        delta = F.softplus(low[:, :RANK] @ p["w_dt"] + p["dt_bias"])
        B, C = low[:, RANK:RANK + N], low[:, RANK + N:]
        s, rows = torch.zeros_like(p["A"]), []
        for t in range(n):
            s = torch.exp(delta[t][:, None] * p["A"]) * s + (delta[t] * c[t])[:, None] * B[t]
            rows.append((s * C[t]).sum(1))
        ys.append(torch.stack(rows) + p["D"] * c)
        lo += n
    y = torch.cat(ys)
    normed = F.rms_norm(y.view(-1, 2, INNER // 2), (INNER // 2,), eps=EPS).reshape(y.shape) * p["w_post"] * F.silu(z)
    return normed @ p["w_out"], h


# Four operators of at most 1.5e-5 each and six fp32 products of up to 48 terms, whose errors each later operator may
# enlarge a few times.
BOUND = 2e-4


def test_block_trains_and_acts():
    need_gpu()
    torch.backends.cuda.matmul.allow_tf32 = False
    lengths = [13, 0, 70, 1, 150]
    t = sum(lengths)
    gen = torch.Generator().manual_seed(3)
    x, residual, dout, dh = (torch.randn(t, DIM, generator=gen).cuda() for _ in range(4))
    ends = torch.from_numpy(ends_of(lengths)).cuda()
    p = _params(0)
    b = Block(t, len(lengths))
    out, h, kept = b.forward(p, x, residual, ends)
    dx, dr, g = b.backward(p, kept, ends, dout, dh)

    q = {k: v.double().cpu().requires_grad_() for k, v in p.items()}
    xs, rs = x.double().cpu().requires_grad_(), residual.double().cpu().requires_grad_()
    want, want_h = _plain(q, xs, rs, lengths)
    ((want * dout.double().cpu()).sum() + (want_h * dh.double().cpu()).sum()).backward()
    check(host(out), want.detach().numpy(), BOUND, "out")
    check(host(h), want_h.detach().numpy(), BOUND, "residual")
    check(host(dx), xs.grad.numpy(), BOUND, "dx")
    check(host(dr), rs.grad.numpy(), BOUND, "dresidual")
    for k in p:
        check(host(g[k]), q[k].grad.numpy(), BOUND, "d" + k)

    # acting: every environment its own state, from nothing, is reading the episodes at once
    n, length = 3, 20
    xe, re = x[:n * length].view(n, length, DIM), residual[:n * length].view(n, length, DIM)
    ends = torch.arange(1, n + 1, device="cuda", dtype=torch.int32) * length
    read, read_h, _ = b.forward(p, xe.reshape(-1, DIM), re.reshape(-1, DIM), ends)
    conv_state, scan_state = torch.zeros(n, INNER, WIDTH - 1, device="cuda"), torch.zeros(n, INNER, N, device="cuda")
    acted = [b.act(p, xe[:, i].contiguous(), re[:, i].contiguous(), conv_state, scan_state) for i in range(length)]
    check(host(torch.stack([a[0] for a in acted], 1).view(-1, DIM)), host(read), BOUND, "acting")
    assert np.array_equal(host(torch.stack([a[1] for a in acted], 1).view(-1, DIM)), host(read_h))
