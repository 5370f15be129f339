"""Workloads of the sequence operators: the gated delta rule over packed episodes and the global gradient norm.

Per value head the gated delta rule keeps a state S [v_dim, k_dim], zero (or given) at an episode's start:

    S_t = a_t S_{t-1} + u_t k_t^T      a_t = exp(g_t)      u_t = beta_t (v_t - a_t S_{t-1} k_t)
    o_t = scale S_t q_t

`kind` says which call a case makes: "act" (one token for each of `slots` environments, states updated in place of
the caller's), "read" (forward over packed episodes), "learn" (forward and backward) and "clip" (the global norm
over many gradient tensors and the clipped gradients).
"""
import math

import torch

own = False

CHUNK = 64
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


def listed():
    seq = dict(k_heads=2, v_heads=2, k_dim=64, v_dim=64, dtype="bf16", states=False)
    return [
        # one environment acts: latency alone
        dict(name="act_one", kind="act", slots=1, k_heads=2, v_heads=2, k_dim=64, v_dim=64, dtype="fp32"),
        # a rack of environments with shared query and key heads
        dict(name="act_rack", kind="act", slots=300, k_heads=4, v_heads=8, k_dim=128, v_dim=128, dtype="bf16"),
        # every environment of a large rollout
        dict(name="act_rollout", kind="act", slots=16384, k_heads=2, v_heads=2, k_dim=64, v_dim=64, dtype="fp32"),
        # 16-step episodes, fp32: the smallest batch
        dict(seq, name="read_tiny", kind="read", episodes=16, shortest=16, longest=16, dtype="fp32"),
        # 64 episodes of 256 steps: the production batch of 16384 transitions
        dict(seq, name="read_production", kind="read", episodes=64, shortest=256, longest=256),
        # odd head sizes, lengths from one step, three value heads a key head, states carried in and out, fp32
        dict(name="read_odd", kind="read", episodes=77, shortest=1, longest=300, k_heads=2, v_heads=6, k_dim=40, v_dim=72,
             dtype="fp32", states=True),
        # one long trajectory, read before acting goes on from its final state
        dict(name="read_long", kind="read", episodes=1, shortest=32768, longest=32768, k_heads=4, v_heads=4, k_dim=128,
             v_dim=128, dtype="bf16", states=True),
        # training on the production batch
        dict(seq, name="learn_production", kind="learn", episodes=64, shortest=256, longest=256),
        dict(seq, name="learn_production_fp32", kind="learn", episodes=64, shortest=256, longest=256, dtype="fp32"),
        # training on about 65536 transitions of episodes of 64 to 512 steps, value heads that share key heads
        dict(name="learn_ragged", kind="learn", episodes=228, shortest=64, longest=512, k_heads=2, v_heads=4, k_dim=128,
             v_dim=128, dtype="bf16", states=False),
        # gradients of a small network: latency
        dict(name="clip_small", kind="clip", tensors=17, elements=120_000, dtype="fp32", ratio=4.0),
        # gradients of a large one
        dict(name="clip_large", kind="clip", tensors=640, elements=150_000_000, dtype="fp32", ratio=4.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    kind = rng.choice(("act", "read", "read", "learn", "learn", "clip"))
    dtype = rng.choice(("fp32", "bf16"))
    if kind == "clip":
        return dict(kind=kind, tensors=_log_int(rng, 1, 640), elements=_log_int(rng, 2000, 100_000_000), dtype=dtype,
                    ratio=rng.choice((0.5, 4.0)))
    k_heads = rng.choice((1, 2, 4))
    v_heads = k_heads * rng.choice((1, 1, 2, 3))
    k_dim, v_dim = (rng.choice((64, 128, 64, 128, 8 * rng.randint(2, 16))) for _ in range(2))
    head = dict(k_heads=k_heads, v_heads=v_heads, k_dim=k_dim, v_dim=v_dim, dtype=dtype)
    if kind == "act":
        return dict(head, kind=kind, slots=_log_int(rng, 1, 4000))
    longest = _log_int(rng, 1, 2048)
    shortest = rng.choice((longest, rng.randint(1, longest)))
    tokens = _log_int(rng, 16, 32768 if dtype == "bf16" else 16384) * 2 // v_heads
    return dict(head, kind=kind, episodes=max(1, 2 * tokens // (shortest + longest)), shortest=shortest, longest=longest,
                states=kind == "read" and rng.random() < 0.3)


def _lengths(case):
    """Whole numbers spread evenly over [shortest, longest] in a fixed mixed order."""
    n, lo, hi = case["episodes"], case["shortest"], case["longest"]
    return [lo + (i * 7919 + 3) % n * (hi - lo) // max(1, n - 1) for i in range(n)]


def _sizes(case):
    """Tensor sizes of a network: two in three are small (biases, norms), odd ones among them."""
    n, total = case["tensors"], case["elements"]
    w = [1.0 if i % 3 == 0 else 0.003 * (1 + i % 7) for i in range(n)]
    s = [max(1, int(total * x / sum(w))) + i % 5 for i, x in enumerate(w)]
    return s


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["kind"] == "clip":
        n = sum(_sizes(case))
        return {"bytes": 2 * n * size + 4, "flops": 3 * n}
    hk, hv, dk, dv = (case[x] for x in ("k_heads", "v_heads", "k_dim", "v_dim"))
    token = size * (2 * hk * dk + 2 * hv * dv + 2 * hv)
    state = 4 * hv * dk * dv
    if case["kind"] == "act":
        return {"bytes": case["slots"] * (token + 2 * state), "flops": case["slots"] * hv * dk * dv * 7}
    t = sum(_lengths(case))
    # the recurrence as it is written: decay, S k, the rank-one update and S q
    forward = t * hv * dk * dv * 7
    if case["kind"] == "read":
        return {"bytes": t * token + case["episodes"] * 2 * state * case["states"], "flops": forward}
    backward = t * size * (2 * hk * dk + 2 * hv * dv + 2 * hv)  # dout read, the five gradients written
    return {"bytes": t * token + backward, "flops": 3 * forward}


def _gates(shape, v_heads, gen):
    """Log decays and write strengths as a gate layer makes them: per-head rates 1 to 16, steps 0.001 to 0.1."""
    rate = 1 + 15 * torch.rand(v_heads, generator=gen, device="cuda")
    step = torch.exp(math.log(0.001) + math.log(100.0) * torch.rand(v_heads, generator=gen, device="cuda"))
    x = 0.5 * torch.randn(*shape, v_heads, generator=gen, device="cuda") + torch.log(torch.expm1(step))
    g = -rate * torch.nn.functional.softplus(x)
    return g, torch.sigmoid(torch.randn(*shape, v_heads, generator=gen, device="cuda"))


def _inputs(case, seed):
    """Inputs alone: q, k and v are slices of one projection's output, as the layer before leaves them."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    if case["kind"] == "clip":
        sizes = _sizes(case)
        n = sum(sizes)
        flat = (torch.randn(n, generator=gen, device="cuda") * (case["ratio"] / math.sqrt(n))).to(dt)
        return dict(flat=flat, sizes=sizes)
    hk, hv, dk, dv = (case[x] for x in ("k_heads", "v_heads", "k_dim", "v_dim"))
    t = case["slots"] if case["kind"] == "act" else sum(_lengths(case))
    act = lambda *s: torch.nn.functional.silu(torch.randn(*s, generator=gen, device="cuda"))  # noqa: E731
    unit = lambda x: x / (x.norm(dim=-1, keepdim=True) + 1e-6)  # noqa: E731
    proj = torch.cat([unit(act(t, hk, dk)).flatten(1), unit(act(t, hk, dk)).flatten(1), act(t, hv * dv)], 1).to(dt)
    q, k, v = proj.split([hk * dk, hk * dk, hv * dv], 1)
    g, beta = _gates((t,), hv, gen)
    s = dict(q=q.unflatten(1, (hk, dk)), k=k.unflatten(1, (hk, dk)), v=v.unflatten(1, (hv, dv)), g=g.to(dt),
             beta=beta.to(dt), scale=dk ** -0.5)
    if case["kind"] == "act" or case["states"]:
        n = case["slots"] if case["kind"] == "act" else case["episodes"]
        s["state"] = 0.3 * torch.randn(n, hv, dv, dk, generator=gen, device="cuda")
    if case["kind"] != "act":
        s["lengths"] = _lengths(case)
        s["ends"] = torch.tensor(s["lengths"]).cumsum(0).to(torch.int32).cuda()
    if case["kind"] == "learn":
        s["dout"] = torch.randn(t, hv, dv, generator=gen, device="cuda").to(dt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    dt = DTYPES[case["dtype"]]
    if case["kind"] == "clip":
        s["grads"] = list(s["flat"].split(s["sizes"]))
        s["flat_out"] = torch.empty_like(s["flat"])
        s["norm"] = torch.empty(1, device="cuda")
        if own:
            import offline_rl_step_gb300 as ofrl

            s["list"] = ofrl.TensorList(s["grads"])
            s["out_list"] = ofrl.TensorList(list(s["flat_out"].split(s["sizes"])))
        return s
    hk, hv, dk, dv = (case[x] for x in ("k_heads", "v_heads", "k_dim", "v_dim"))
    t = s["q"].shape[0]
    new = lambda *shape: torch.empty(*shape, device="cuda", dtype=dt)  # noqa: E731
    s["out"] = new(t, hv, dv)
    if "state" in s:
        s["new_state"] = torch.empty_like(s["state"])
    if case["kind"] == "learn":
        s["grads"] = [new(t, hk, dk), new(t, hk, dk), new(t, hv, dv), new(t, hv), new(t, hv)]
    if own:
        import offline_rl_step_gb300 as ofrl

        rows = case["slots"] if case["kind"] == "act" else case["episodes"]
        s["ctx"] = ofrl.DeltaRule(hk, hv, dk, dv, case["dtype"], max_tokens=t, max_episodes=rows)
        if case["kind"] == "learn":
            s["saved"] = s["ctx"].saved(t, rows)
    return s


def run(s):
    kind = s["case"]["kind"]
    if not own:
        return _plain(s)
    import offline_rl_step_gb300 as ofrl

    if kind == "clip":
        ofrl.global_norm_clip(s["list"], 1.0, s["norm"], out=s["out_list"])
        return {"norm": s["norm"], "grads": s["flat_out"]}
    tokens = [s[x] for x in ("q", "k", "v", "g", "beta")]
    if kind == "act":
        ofrl.delta_step(s["ctx"], *tokens, s["state"], s["out"], scale=s["scale"], new_state=s["new_state"])
        return {"out": s["out"], "state": s["new_state"]}
    ofrl.delta_forward(s["ctx"], *tokens, s["ends"], s["out"], scale=s["scale"], init_state=s.get("state"),
                       final_state=s.get("new_state"), saved=s.get("saved"))
    if kind == "read":
        return {"out": s["out"], "state": s.get("new_state")}
    ofrl.delta_backward(s["ctx"], *tokens, s["ends"], s["saved"], s["dout"], *s["grads"], scale=s["scale"])
    return {"out": s["out"], "grads": s["grads"]}


# ---- the plain form: chunks of 64 tokens, 32 bits throughout -------------------------------------------------------


def _plain(s):
    kind, dt = s["case"]["kind"], DTYPES[s["case"]["dtype"]]
    if kind == "clip":
        flat = torch.cat([x.reshape(-1).float() for x in s["grads"]])
        norm = flat.square().sum().sqrt()
        factor = torch.where(norm > 1.0, 1.0 / norm, torch.ones_like(norm))
        return {"norm": norm.reshape(1), "grads": (flat * factor).to(dt)}
    if kind == "act":
        return _plain_step(s, dt)
    return _plain_sequence(s, dt)


def _plain_step(s, dt):
    group = s["v"].shape[1] // s["k"].shape[1]
    q, k = (s[x].float().repeat_interleave(group, 1) for x in ("q", "k"))
    v, g, beta = (s[x].float() for x in ("v", "g", "beta"))
    state = s["state"] * g.exp()[..., None, None]
    u = beta[..., None] * (v - (state * k[..., None, :]).sum(-1))
    state = state + u[..., None] * k[..., None, :]
    return {"out": (s["scale"] * (state * q[..., None, :]).sum(-1)).to(dt), "state": state}


def _chunks(x, index, valid):
    """[tokens, heads, ...] to [episodes, heads, chunks, CHUNK, ...], zero past an episode's end."""
    x = x.float()[index] * valid.reshape(*valid.shape, *[1] * (x.dim() - 1))
    return x.movedim(2, 1).unflatten(2, (-1, CHUNK))


def _tokens(x, index, valid, t):
    """The inverse of _chunks."""
    x = x.flatten(2, 3).movedim(1, 2)
    out = x.new_empty(t, *x.shape[2:])
    out[index[valid]] = x[valid]
    return out


def _plain_sequence(s, dt):
    t, group = s["q"].shape[0], s["v"].shape[1] // s["k"].shape[1]
    longest = -(-max(s["lengths"]) // CHUNK) * CHUNK
    ends = s["ends"].long()
    starts = torch.cat([ends.new_zeros(1), ends[:-1]])
    at = starts[:, None] + torch.arange(longest, device="cuda")
    valid = at < ends[:, None]
    index = torch.where(valid, at, 0)
    q, k, v, g, b = (_chunks(s[x], index, valid) for x in ("q", "k", "v", "g", "beta"))
    q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
    q = q * s["scale"]
    n, h, chunks, c, dk = k.shape
    lower = torch.ones(c, c, device="cuda", dtype=torch.bool).tril()
    cum = g.cumsum(-1)
    decay = torch.where(lower, cum[..., :, None] - cum[..., None, :], -math.inf).exp()
    gam, rest = cum.exp()[..., None], (cum[..., -1:] - cum).exp()[..., None]
    last = gam[..., -1:, :]
    kk = (k @ k.mT) * decay * lower.tril(-1)
    a = b[..., None] * kk
    inv = torch.eye(c, device="cuda").expand_as(a).clone()  # (1 + a)^-1 by forward substitution
    for i in range(1, c):
        inv[..., i, :i] = -(a[..., i, None, :i] @ inv[..., :i, :i])[..., 0, :]
    p = (q @ k.mT) * decay
    gk = gam * k
    w, y = inv @ (b[..., None] * gk), inv @ (b[..., None] * v)
    state = s["state"].mT if "state" in s else torch.zeros(n, h, dk, v.shape[-1], device="cuda")
    u, before = torch.empty_like(v), torch.empty(chunks if "dout" in s else 0, *state.shape, device="cuda")
    rk = rest * k
    for i in range(chunks):
        if "dout" in s:
            before[i] = state
        u[:, :, i] = y[:, :, i] - w[:, :, i] @ state
        v[:, :, i] -= gk[:, :, i] @ state  # from here on v less what the state predicts
        y[:, :, i] = (gam[:, :, i] * q[:, :, i]) @ state + p[:, :, i] @ u[:, :, i]
        state = last[:, :, i] * state + rk[:, :, i].mT @ u[:, :, i]
    out = _tokens(y, index, valid, t).to(dt)
    if "dout" not in s:
        return {"out": out, "state": state.mT.contiguous() if "state" in s else None}
    do = _chunks(s["dout"], index, valid)
    x = v
    du = p.mT @ do
    dx, dend, dlast = torch.empty_like(x), torch.empty_like(before), torch.zeros_like(state)
    gq = gam * q
    for i in range(chunks - 1, -1, -1):
        dend[i] = dlast
        du[:, :, i] += rk[:, :, i] @ dlast
        dx[:, :, i] = b[:, :, i, :, None] * (inv[:, :, i].mT @ du[:, :, i])
        dlast = last[:, :, i] * dlast + gq[:, :, i].mT @ do[:, :, i] - gk[:, :, i].mT @ dx[:, :, i]
    before, dend = before.movedim(0, 2), dend.movedim(0, 2)
    r = inv.mT @ du
    dp, da = (do @ u.mT) * lower, -(r @ u.mT) * lower.tril(-1)
    dpd, m = dp * decay, b[..., None] * da * decay
    from_state_q, from_state_k = gam * (do @ before.mT), -gam * (dx @ before.mT)
    to_state_k = rest * (u @ dend.mT)
    dq = from_state_q + dpd @ k
    row, col = from_state_k + m @ k, dpd.mT @ q + m.mT @ k + to_state_k
    db = (r * x).sum(-1) + (da * kk).sum(-1)
    pairs = dp * p + da * a
    dcum = (from_state_q * q + from_state_k * k - to_state_k * k).sum(-1) + pairs.sum(-1) - pairs.sum(-2)
    dcum[..., -1] += (to_state_k * k).sum((-1, -2)) + last[..., 0, 0] * (before * dend).sum((-1, -2))
    dg = dcum.flip(-1).cumsum(-1).flip(-1)
    dq, dk_ = (z.unflatten(1, (-1, group)).sum(2) for z in (s["scale"] * dq, row + col))
    return {"out": out, "grads": [_tokens(z, index, valid, t).to(dt) for z in (dq, dk_, dx, dg, db)]}


# ---- 64 bits: the recurrence token by token, and its adjoint --------------------------------------------------------


def exact(case, seed):
    s = _inputs(case, seed)
    if case["kind"] == "clip":
        flat = s["flat"].double()
        norm = torch.linalg.vector_norm(flat)
        return {"norm": norm.reshape(1), "grads": flat / norm.clamp(min=1.0)}
    group = s["v"].shape[1] // s["k"].shape[1]
    q, k, v, g, beta = (s[x].double() for x in ("q", "k", "v", "g", "beta"))
    q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
    if case["kind"] == "act":
        lengths, starts = [1] * case["slots"], list(range(case["slots"]))
    else:
        lengths = s["lengths"]
        starts = [sum(lengths[:i]) for i in range(len(lengths))]
    t, h, dv = v.shape
    learn = case["kind"] == "learn"
    state = s["state"].double() if "state" in s else torch.zeros(len(lengths), h, dv, k.shape[-1], device="cuda", dtype=torch.float64)
    order = sorted(range(len(lengths)), key=lambda i: -lengths[i])  # the episodes still running come first
    state = state[order]
    first = torch.tensor([starts[i] for i in order], device="cuda")
    out, kept = torch.empty_like(v), []
    for i in range(max(lengths)):
        n = sum(x > i for x in lengths)
        at = first[:n] + i
        ki, a = k[at], g[at].exp()[..., None, None]
        if learn:
            kept.append(state[:n].clone())
        old = a * state[:n]
        u = beta[at][..., None] * (v[at] - torch.einsum("nhvk,nhk->nhv", old, ki))
        state[:n] = old + torch.einsum("nhv,nhk->nhvk", u, ki)
        out[at] = s["scale"] * torch.einsum("nhvk,nhk->nhv", state[:n], q[at])
    back = torch.empty_like(state)
    back[order] = state
    if not learn:
        return {"out": out, "state": back if "state" in s else None}
    do = s["dout"].double()
    dq, dk, dval, dg, db = (torch.zeros_like(x) for x in (q, k, v, g, beta))
    ds = torch.zeros_like(state)
    for i in range(max(lengths) - 1, -1, -1):
        n = sum(x > i for x in lengths)
        at = first[:n] + i
        qi, ki, a, bi = q[at], k[at], g[at].exp()[..., None, None], beta[at][..., None]
        old = a * kept.pop()
        err = v[at] - torch.einsum("nhvk,nhk->nhv", old, ki)
        u = bi * err
        d, doi = ds[:n], s["scale"] * do[at]
        dq[at] = torch.einsum("nhvk,nhv->nhk", old + torch.einsum("nhv,nhk->nhvk", u, ki), doi)
        d = d + torch.einsum("nhv,nhk->nhvk", doi, qi)
        du = torch.einsum("nhvk,nhk->nhv", d, ki)
        db[at] = (du * err).sum(-1)
        dval[at] = bi * du
        dk[at] = torch.einsum("nhvk,nhv->nhk", d, u) - torch.einsum("nhvk,nhv->nhk", old, bi * du)
        dold = d - torch.einsum("nhv,nhk->nhvk", bi * du, ki)
        dg[at] = (dold * old).sum((-1, -2))
        ds[:n] = a * dold
    dq, dk = (z.unflatten(1, (-1, group)).sum(2) for z in (dq, dk))
    return {"out": out, "grads": [dq, dk, dval, dg, db]}
