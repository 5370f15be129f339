"""A value head with a memory: trained over packed episodes, then acting one step at a time.

Every episode shows a sign in its first step only, and the value of every later step is that sign: what a value
network on single states cannot learn.  The memory is the gated delta rule.  One training step:

    projections -> delta_forward -> read-out -> expectile_loss -> delta_backward -> projections' gradients
    -> global_norm over all gradients -> adam_step for each parameter, clipped by that norm

Acting takes the trained parameters and delta_step, whose state is all that is kept of an environment's past.

    python examples/episode_memory.py
"""
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import offline_rl_step_gb300 as ofrl  # noqa: E402


class _Delta(torch.autograd.Function):
    @staticmethod
    def forward(fn, rule, ends, q, k, v, g, beta):
        saved = rule.saved(q.shape[0], ends.numel())
        out = torch.empty(q.shape[0], rule.v_heads, rule.v_dim, device=q.device, dtype=rule.dtype)
        ofrl.delta_forward(rule, q, k, v, g, beta, ends, out, saved=saved)
        fn.rule = rule
        fn.save_for_backward(ends, saved, q, k, v, g, beta)
        return out

    @staticmethod
    def backward(fn, dout):
        ends, saved, q, k, v, g, beta = fn.saved_tensors
        grads = [torch.empty_like(t, memory_format=torch.contiguous_format) for t in (q, k, v, g, beta)]
        ofrl.delta_backward(fn.rule, q, k, v, g, beta, ends, saved, dout.contiguous(), *grads)
        return (None, None, *grads)


class Memory:
    """States [tokens, state_dim] -> values [tokens], through the gated delta rule."""

    def __init__(self, state_dim: int, heads: int = 2, dim: int = 64, max_tokens: int = 16384, max_episodes: int = 1024,
                 seed: int = 0):
        gen = torch.Generator().manual_seed(seed)
        self.heads, self.dim = heads, dim
        self.rule = ofrl.DeltaRule(heads, heads, dim, dim, "bf16", max_tokens, max_episodes)
        new = lambda *s: (torch.randn(*s, generator=gen) * s[0] ** -0.5).cuda()  # noqa: E731
        self.w_in, self.w_gate, self.w_out = new(state_dim, 3 * heads * dim), new(state_dim, 2 * heads), new(heads * dim)
        # decays near one, write strengths near a half
        self.b_gate = torch.cat([torch.full((heads,), -4.0), torch.zeros(heads)]).cuda()
        self.params = [self.w_in, self.w_gate, self.w_out, self.b_gate]
        for p in self.params:
            p.requires_grad_()
            p.grad = torch.zeros_like(p)
        self.grads = ofrl.TensorList([p.grad for p in self.params])
        self.moments = [(torch.zeros_like(p), torch.zeros_like(p)) for p in self.params]
        self.norm = torch.zeros(1, device="cuda")
        self.t = 0

    def tokens(self, x):
        """What the rule takes: unit queries and keys, values, log decays and write strengths."""
        q, k, v = (x @ self.w_in).unflatten(1, (3 * self.heads, self.dim)).split(self.heads, 1)
        g, beta = (x @ self.w_gate + self.b_gate).split(self.heads, 1)
        dt = self.rule.dtype
        return (F.normalize(q, dim=-1).to(dt), F.normalize(k, dim=-1).to(dt), v.to(dt), (-F.softplus(g)).to(dt),
                torch.sigmoid(beta).to(dt))

    def read_out(self, out):
        return out.flatten(1).float() @ self.w_out

    def values(self, x, episode_ends):
        return self.read_out(_Delta.apply(self.rule, episode_ends, *self.tokens(x)))

    def train_step(self, ctx, x, episode_ends, target, opt, tau=0.5):
        """One update; returns the loss (device scalar) before it."""
        v = self.values(x, episode_ends)
        loss, dv = torch.empty(1, device="cuda"), torch.empty_like(v)
        ofrl.expectile_loss(ctx, target, v.detach(), tau, loss, dv)
        for p in self.params:
            p.grad.zero_()
        v.backward(dv)
        ofrl.global_norm(self.grads, self.norm)
        self.t += 1
        for p, (m, s) in zip(self.params, self.moments):
            ofrl.adam_step(ctx, p.detach(), p.grad, m, s, self.t, opt, grad_norm=self.norm)
        return loss

    @torch.no_grad()
    def act(self, x, state):
        """Values of one step in every environment; state [environments, heads, dim, dim] moves on in place."""
        out = torch.empty(x.shape[0], self.heads, self.dim, device="cuda", dtype=self.rule.dtype)
        ofrl.delta_step(self.rule, *self.tokens(x), state, out)
        return self.read_out(out)


def episodes(n, length, state_dim, gen):
    """States [n, length, state_dim] and the signs.  Features 0 and 1: the sign and a mark, in step 0 only; feature 2
    is one throughout, the rest is noise."""
    x = 0.3 * torch.randn(n, length, state_dim, generator=gen, device="cuda")
    sign = torch.randint(0, 2, (n,), generator=gen, device="cuda") * 2.0 - 1.0
    x[:, :, :2] = 0.0
    x[:, 0, 0], x[:, 0, 1] = sign, 1.0
    x[:, :, 2] = 1.0
    return x, sign


def main(steps=200, n=64, length=256, state_dim=16, seed=0, say=print):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ctx = ofrl.Context(state_dim, 64, 4, max_batch=n * length)
    mem = Memory(state_dim, max_tokens=n * length, max_episodes=n)
    opt = ofrl.Opt(lr=1e-2, max_grad_norm=1.0)
    ends = torch.arange(1, n + 1, device="cuda", dtype=torch.int32) * length
    losses = []
    for i in range(steps):
        x, sign = episodes(n, length, state_dim, gen)
        target = sign[:, None].expand(n, length).flatten().contiguous()
        losses.append(mem.train_step(ctx, x.flatten(0, 1), ends, target, opt))
        if i % 50 == 0 or i == steps - 1:
            say(f"step {i}: loss {losses[-1].item():.4f}, gradient norm {mem.norm.item():.4f}")
    # the same memory, acting: one step at a time against the whole episode at once
    x, sign = episodes(n, length, state_dim, gen)
    with torch.no_grad():
        read = mem.values(x.flatten(0, 1), ends).view(n, length)
    state = torch.zeros(n, mem.heads, mem.dim, mem.dim, device="cuda")
    acted = torch.stack([mem.act(x[:, i], state) for i in range(length)], 1)
    right = (acted[:, -1].sign() == sign).float().mean().item()
    say(f"acting: {100 * right:.1f}% of {n} episodes end with the right sign, "
        f"largest difference from reading at once {(acted - read).abs().max().item():.4f}")
    status = mem.rule.poll_status()
    return [x.item() for x in losses], acted, read, right, status


if __name__ == "__main__":
    main()
