"""Workloads of a state space block: short causal convolution, selective scan, gated norm and residual norm.

`op` says which operator a case runs, `kind` which call: "act" (one token for each of `slots` environments, states
written to a second buffer), "read" (forward), "learn" (forward and backward).  Tokens are the packed transitions of
episodes; per channel d and state n

    conv:      pre_t = bias + sum_j w_j x_{t-W+1+j}          out = silu(pre)
    scan:      h_t = exp(delta_t A) h_{t-1} + delta_t B_t x_t     out = (sum_n C_t h_t + D x_t) silu(z_t)
               delta = softplus(dt + dt_bias)
    gated:     out = w x / rms(x) silu(z)        (or the norm of x silu(z), "gate_first")
    residual:  h = residual + scale x            out = w h / rms(h)
"""
import math

import torch

own = False

CHUNK = 64
EPS = 1e-5
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # 300 environments act: one token through the convolution, latency
        dict(name="conv_act", op="conv", kind="act", slots=300, channels=256, width=4, dtype="bf16"),
        # ragged episodes from one step on, fp32, an odd channel count, states carried in and out
        dict(name="conv_read_odd", op="conv", kind="read", episodes=77, shortest=1, longest=300, channels=360, width=3,
             dtype="fp32", states=True),
        # training on about 65536 transitions of 64 to 512 steps
        dict(name="conv_learn", op="conv", kind="learn", episodes=228, shortest=64, longest=512, channels=1024, width=4,
             dtype="bf16", states=False),
        # every environment of a large rollout
        dict(name="scan_act_rollout", op="scan", kind="act", slots=16384, channels=256, state=16, groups=1, dtype="bf16",
             gate=True),
        # odd channels and states, lengths from one step, fp32, two groups, no gate, states carried in and out
        dict(name="scan_read_odd", op="scan", kind="read", episodes=77, shortest=1, longest=300, channels=144, state=12,
             groups=2, dtype="fp32", gate=False, states=True),
        # one long trajectory, read before acting goes on from its final state
        dict(name="scan_read_long", op="scan", kind="read", episodes=1, shortest=32768, longest=32768, channels=1024,
             state=16, groups=1, dtype="bf16", gate=True, states=True),
        # the production batch of 16384 transitions, 64 episodes of 256 steps, trained in fp32
        dict(name="scan_learn_production", op="scan", kind="learn", episodes=64, shortest=256, longest=256, channels=128,
             state=16, groups=1, dtype="fp32", gate=True, states=False),
        # training on about 65536 transitions of 64 to 512 steps
        dict(name="scan_learn_ragged", op="scan", kind="learn", episodes=228, shortest=64, longest=512, channels=512,
             state=16, groups=1, dtype="bf16", gate=True, states=False),
        # heads of 64 channels normed apart, fp32, the smallest batch
        dict(name="gated_read", op="gated", kind="read", rows=256, channels=128, groups=2, dtype="fp32", gate_first=False),
        # training on 65536 transitions, the whole row normed
        dict(name="gated_learn", op="gated", kind="learn", rows=65536, channels=1024, groups=1, dtype="bf16",
             gate_first=True),
        # odd rows, the residual stream kept in fp32 beside bf16 blocks
        dict(name="residual_read", op="residual", kind="read", rows=5003, channels=760, dtype="bf16", residual="fp32",
             scale=True),
        # training on 65536 transitions
        dict(name="residual_learn", op="residual", kind="learn", rows=65536, channels=1024, dtype="bf16", residual="bf16",
             scale=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _lengths_of(rng, tokens):
    longest = _log_int(rng, 1, 4096)
    shortest = rng.choice((longest, rng.randint(1, longest)))
    return dict(episodes=max(1, 2 * tokens // (shortest + longest)), shortest=shortest, longest=longest)


def draw(rng):
    op = rng.choice(("conv", "scan", "scan", "gated", "residual"))
    dtype = rng.choice(("fp32", "bf16"))
    if op == "gated" or op == "residual":
        kind = rng.choice(("read", "learn"))
        rows, groups = _log_int(rng, 1, 65536), 1
        channels = 8 * _log_int(rng, 1, 512)
        if op == "gated":
            groups = rng.choice((1, 1, 2, 4))
            channels *= groups
        rows = max(1, min(rows, 2 ** 26 // channels))
        if op == "gated":
            return dict(op=op, kind=kind, rows=rows, channels=channels, groups=groups, dtype=dtype,
                        gate_first=rng.random() < 0.5)
        return dict(op=op, kind=kind, rows=rows, channels=channels, dtype=dtype, residual=rng.choice(("fp32", dtype)),
                    scale=rng.random() < 0.7)
    kind = rng.choice(("act", "read", "learn"))
    if op == "conv":
        channels = 8 * _log_int(rng, 1, 256)
        case = dict(op=op, kind=kind, channels=channels, width=rng.choice((2, 3, 4, 4)), dtype=dtype)
        if kind == "act":
            return dict(case, slots=_log_int(rng, 1, 16384))
        tokens = min(_log_int(rng, 16, 65536), 2 ** 25 // channels)
        return dict(case, **_lengths_of(rng, tokens), states=kind == "read" and rng.random() < 0.3)
    groups = rng.choice((1, 1, 1, 2, 4))
    state = rng.choice((16, 16, 16, 4, 8, 32, 64, 4 * rng.randint(1, 16)))
    channels = groups * 8 * _log_int(rng, 1, 128 // groups)
    case = dict(op=op, kind=kind, channels=channels, state=state, groups=groups, dtype=dtype, gate=rng.random() < 0.7)
    if kind == "act":
        return dict(case, slots=_log_int(rng, 1, min(16384, 2 ** 27 // (channels * state))))
    tokens = min(_log_int(rng, 16, 65536 if dtype == "bf16" else 32768), 2 ** 28 // (channels * state))
    return dict(case, **_lengths_of(rng, max(1, tokens)), states=kind == "read" and rng.random() < 0.3)


def _lengths(case):
    """Whole numbers spread evenly over [shortest, longest] in a fixed mixed order."""
    n, lo, hi = case["episodes"], case["shortest"], case["longest"]
    return [lo + (i * 7919 + 3) % n * (hi - lo) // max(1, n - 1) for i in range(n)]


def _rows(case):
    if case["kind"] == "act":
        return case["slots"]
    return case["rows"] if "rows" in case else sum(_lengths(case))


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    op, learn, act = case["op"], case["kind"] == "learn", case["kind"] == "act"
    t, d = _rows(case), case["channels"]
    states = case["slots"] if act else case["episodes"] if case.get("states") else 0
    if op == "conv":
        w = case["width"]
        return {"bytes": size * t * d * (4 if learn else 2) + 4 * d * (w + 1) * (1 + learn) + 2 * states * size * d * (w - 1),
                "flops": t * d * (2 * w + 4 + (4 * w + 8) * learn)}
    if op == "scan":
        n, g, gate = case["state"], case["groups"], case["gate"]
        tokens = size * t * (3 * d + gate * d + 2 * g * n)
        # the gradient of the output read, those of the five inputs written
        grads = (size * t * (3 * d + gate * d + 2 * g * n) + 4 * d * (n + 2)) * learn
        # the recurrence as it is written: delta A, exp, a h, delta x B, its sum, C h, its sum; its adjoint has 16
        return {"bytes": tokens + grads + 4 * d * (n + 2) + 2 * states * 4 * d * n, "flops": t * d * n * (7 + 16 * learn)}
    if op == "gated":
        return {"bytes": size * t * d * (3 + 3 * learn) + 4 * d * (1 + learn), "flops": t * d * (9 + 20 * learn)}
    res = 4 if case["residual"] == "fp32" else 2
    return {"bytes": t * d * (2 * size + 2 * res + (2 * size + 2 * res) * learn) + 8 * d * (1 + learn),
            "flops": t * d * (6 + 12 * learn)}


def _inputs(case, seed):
    """Inputs alone, as the layers before leave them: slices of one projection's output where they are that."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    uni = lambda *s: torch.rand(*s, generator=gen, device="cuda")  # noqa: E731
    op, t, d = case["op"], _rows(case), case["channels"]
    s = {}
    if op in ("conv", "scan"):
        s["lengths"] = [1] * t if case["kind"] == "act" else _lengths(case)
        s["ends"] = torch.tensor(s["lengths"]).cumsum(0).to(torch.int32).cuda()
    states = case["kind"] == "act" or case.get("states")
    if op == "conv":
        w = case["width"]
        s["x"] = rand(t, 2 * d).to(dt)[:, :d]
        s["weight"], s["bias"] = (2 * uni(d, w) - 1) * w ** -0.5, (2 * uni(d) - 1) * w ** -0.5
        if states:
            s["state"] = rand(len(s["lengths"]), d, w - 1).to(dt)
    elif op == "scan":
        n, g = case["state"], case["groups"]
        s["x"] = torch.nn.functional.silu(rand(t, d)).to(dt)
        s["z"] = rand(t, 2 * d).to(dt)[:, d:] if case["gate"] else None
        # steps 0.001 to 0.1 a channel, decays -1 .. -N as they are initialised, moved a little
        step = torch.exp(math.log(0.001) + math.log(100.0) * uni(d))
        s["dt"], s["dt_bias"] = (0.5 * rand(t, d)).to(dt), torch.log(torch.expm1(step))
        s["A"] = -torch.arange(1, n + 1, device="cuda") * torch.exp(0.1 * rand(d, n))
        bc = rand(t, 8 + 2 * g * n).to(dt)
        s["B"], s["C"] = (x.unflatten(1, (g, n)) for x in bc[:, 8:].split(g * n, 1))
        s["D"] = 1 + 0.1 * rand(d)
        if states:
            s["state"] = 0.3 * rand(len(s["lengths"]), d, n)
    elif op == "gated":
        s["x"], s["z"] = (1.5 * rand(t, d)).to(dt), rand(t, 2 * d).to(dt)[:, d:]
        s["weight"] = 1 + 0.2 * rand(d)
    else:
        s["x"], s["residual"] = rand(t, d).to(dt), (2 * rand(t, d)).to(DTYPES[case["residual"]])
        s["weight"], s["scale"] = 1 + 0.2 * rand(d), 0.1 + 0.05 * rand(d) if case["scale"] else None
    if case["kind"] == "learn":
        s["dout"] = rand(t, d).to(dt)
        if op == "residual":
            s["dres"] = rand(t, d).to(DTYPES[case["residual"]])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    dt, t, d, op, learn = DTYPES[case["dtype"]], _rows(case), case["channels"], case["op"], case["kind"] == "learn"
    new = lambda *shape, dtype=dt: torch.empty(*shape, device="cuda", dtype=dtype)  # noqa: E731
    f32 = torch.float32
    s["out"] = new(t, d)
    if "state" in s:
        s["new_state"] = torch.empty_like(s["state"])
    if op == "residual":
        s["res_out"] = torch.empty_like(s["residual"])
    if learn and op == "conv":
        s["grads"] = {"x": new(t, d), "weight": new(d, case["width"], dtype=f32), "bias": new(d, dtype=f32)}
    if learn and op == "scan":
        n, g = case["state"], case["groups"]
        s["grads"] = {"x": new(t, d), "dt": new(t, d), "B": new(t, g, n), "C": new(t, g, n), "A": new(d, n, dtype=f32),
                      "D": new(d, dtype=f32), "dt_bias": new(d, dtype=f32), "z": new(t, d) if case["gate"] else None}
    if learn and op == "gated":
        s["grads"] = {"x": new(t, d), "z": new(t, d), "weight": new(d, dtype=f32)}
    if learn and op == "residual":
        s["grads"] = {"x": new(t, d), "residual": torch.empty_like(s["residual"]), "weight": new(d, dtype=f32),
                      "scale": new(d, dtype=f32) if case["scale"] else None}
    if own:
        import offline_rl_step_gb300 as ofrl

        if op == "conv":
            s["ctx"] = ofrl.CausalConv(d, case["width"], "silu", case["dtype"], max_tokens=t,
                                       max_episodes=len(s["lengths"]), backward=learn)
        elif op == "scan":
            s["ctx"] = ofrl.SelectiveScan(d, case["state"], case["groups"], case["dtype"], max_tokens=t,
                                          max_episodes=len(s["lengths"]), backward=learn)
            if learn:
                s["saved"] = s["ctx"].saved(t)
        else:
            s["ctx"] = ofrl.BlockNorm(d, case.get("groups", 1), case["dtype"], case.get("residual"), backward=learn)
    return s


def run(s):
    if not own:
        return PLAIN[s["case"]["op"]](s)
    import offline_rl_step_gb300 as ofrl

    case, ctx = s["case"], s["ctx"]
    op, kind, g = case["op"], case["kind"], s.get("grads")
    if op == "conv":
        if kind == "act":
            ofrl.conv_step(ctx, s["x"], s["weight"], s["state"], s["out"], bias=s["bias"], new_state=s["new_state"])
            return {"out": s["out"], "state": s["new_state"]}
        ofrl.conv_forward(ctx, s["x"], s["weight"], s["ends"], s["out"], bias=s["bias"], init_state=s.get("state"),
                          final_state=s.get("new_state"))
        if kind == "read":
            return {"out": s["out"], "state": s.get("new_state")}
        ofrl.conv_backward(ctx, s["x"], s["weight"], s["ends"], s["dout"], g["x"], g["weight"], bias=s["bias"],
                           dbias=g["bias"])
    elif op == "scan":
        tokens = [s[x] for x in ("x", "dt", "A", "B", "C")]
        more = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
        if kind == "act":
            ofrl.scan_step(ctx, *tokens, s["state"], s["out"], new_state=s["new_state"], **more)
            return {"out": s["out"], "state": s["new_state"]}
        ofrl.scan_forward(ctx, *tokens, s["ends"], s["out"], init_state=s.get("state"), final_state=s.get("new_state"),
                          saved=s.get("saved"), **more)
        if kind == "read":
            return {"out": s["out"], "state": s.get("new_state")}
        ofrl.scan_backward(ctx, *tokens, s["ends"], s["saved"], s["dout"], g["x"], g["dt"], g["A"], g["B"], g["C"],
                           dD=g["D"], dz=g["z"], ddt_bias=g["dt_bias"], **more)
    elif op == "gated":
        ofrl.gated_norm(ctx, s["x"], s["z"], s["weight"], s["out"], eps=EPS, gate_first=case["gate_first"])
        if kind == "learn":
            ofrl.gated_norm_backward(ctx, s["x"], s["z"], s["weight"], s["dout"], g["x"], g["z"], g["weight"], eps=EPS,
                                     gate_first=case["gate_first"])
    else:
        ofrl.residual_norm(ctx, s["x"], s["residual"], s["weight"], s["res_out"], s["out"], scale=s["scale"], eps=EPS)
        if kind == "learn":
            ofrl.residual_norm_backward(ctx, s["x"], s["residual"], s["weight"], s["dout"], g["x"], g["residual"],
                                        g["weight"], scale=s["scale"], dscale=g["scale"], d_residual_out=s["dres"], eps=EPS)
    out = {"out": s["out"]}
    if op == "residual":
        out["residual"] = s["res_out"]
    if kind == "learn":
        out["grads"] = g
    return out


# ---- the plain forms: 32 bits throughout, rounded once at the end --------------------------------------------------


def _sig(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _softplus(x):
    return x.clamp(min=0.0) + torch.log1p(torch.exp(-x.abs()))


def _spread(s, multiple):
    """Index [episodes, longest] of each token and whether there is one."""
    longest = -(-max(s["lengths"]) // multiple) * multiple
    ends = s["ends"].long()
    at = (ends - torch.tensor(s["lengths"], device="cuda"))[:, None] + torch.arange(longest, device="cuda")
    valid = at < ends[:, None]
    return torch.where(valid, at, 0), valid


def _pack(x, index, valid, t):
    """[episodes, longest, ...] to [tokens, ...]."""
    out = x.new_empty(t, *x.shape[2:])
    out[index[valid]] = x[valid]
    return out


def _plain_conv(s):
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    w, t, d, k = s["weight"], *s["x"].shape, case["width"]
    if case["kind"] == "act":
        seen = torch.cat([s["state"].float(), s["x"].float()[:, :, None]], 2)
        pre = s["bias"] + (seen * w).sum(-1)
        return {"out": (pre * _sig(pre)).to(dt), "state": seen[:, :, 1:].to(dt)}
    index, valid = _spread(s, 1)
    n, longest = index.shape
    x = s["x"].float()[index] * valid[..., None]
    before = s["state"].float().mT if "state" in s else x.new_zeros(n, k - 1, d)
    x = torch.cat([before, x], 1)
    pre = s["bias"] + sum(x[:, j:j + longest] * w[:, j] for j in range(k))
    sig = _sig(pre)
    result = {"out": _pack(pre * sig, index, valid, t).to(dt)}
    if case["kind"] == "read":
        last = torch.tensor(s["lengths"], device="cuda")[:, None] + torch.arange(k - 1, device="cuda")
        result["state"] = (x[torch.arange(n, device="cuda")[:, None], last].mT.contiguous().to(dt) if "state" in s
                           else None)
        return result
    dpre = s["dout"].float()[index] * valid[..., None] * sig * (1.0 + pre * (1.0 - sig))
    dx = torch.zeros_like(x)
    for j in range(k):
        dx[:, j:j + longest] += dpre * w[:, j]
    result["grads"] = {"x": _pack(dx[:, k - 1:], index, valid, t).to(dt),
                       "weight": torch.stack([(dpre * x[:, j:j + longest]).sum((0, 1)) for j in range(k)], 1),
                       "bias": dpre.sum((0, 1))}
    return result


def _plain_scan(s):
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    t, d = s["x"].shape
    group = d // case["groups"]
    A = s["A"]
    if case["kind"] == "act":
        x, z = s["x"].float(), s["z"].float() if case["gate"] else None
        delta = _softplus(s["dt"].float() + s["dt_bias"])
        b, c = (s[i].float().repeat_interleave(group, 1) for i in ("B", "C"))
        h = torch.exp(delta[..., None] * A) * s["state"] + (delta * x)[..., None] * b
        y = (h * c).sum(-1) + s["D"] * x
        return {"out": (y * z * _sig(z) if case["gate"] else y).to(dt), "state": h}
    index, valid = _spread(s, CHUNK)
    chunks = lambda x: (x.float()[index] * valid.reshape(*valid.shape, *[1] * (x.dim() - 1))).unflatten(1, (-1, CHUNK))  # noqa: E731
    x, raw, b, c = (chunks(s[i]) for i in ("x", "dt", "B", "C"))
    z = chunks(s["z"]) if case["gate"] else None
    raw = raw + s["dt_bias"]
    delta = _softplus(raw) * valid.unflatten(1, (-1, CHUNK))[..., None]
    dx = delta * x
    n, nc = x.shape[:2]
    bs = [b[:, :, i].repeat_interleave(group, 2) for i in range(CHUNK)]
    cs = [c[:, :, i].repeat_interleave(group, 2) for i in range(CHUNK)]
    decay = lambda i: torch.exp(delta[:, :, i, :, None] * A)  # noqa: E731
    # every chunk from a zero state, then the states between chunks
    h = x.new_zeros(n, nc, d, case["state"])
    for i in range(CHUNK):
        h = decay(i) * h + dx[:, :, i, :, None] * bs[i]
    total = delta.sum(2)[..., None]
    start = torch.empty_like(h)
    carry = s["state"] if "state" in s else torch.zeros_like(h[:, 0])
    for j in range(nc):
        start[:, j] = carry
        carry = torch.exp(total[:, j] * A) * carry + h[:, j]
    h, hs, y = start, [], torch.empty_like(x)
    for i in range(CHUNK):
        if case["kind"] == "learn":
            hs.append(h)
        h = decay(i) * h + dx[:, :, i, :, None] * bs[i]
        y[:, :, i] = (h * cs[i]).sum(-1)
    y += s["D"] * x
    out = y * z * _sig(z) if case["gate"] else y
    result = {"out": _pack(out.flatten(1, 2), index, valid, t).to(dt)}
    if case["kind"] == "read":
        result["state"] = carry if "state" in s else None
        return result
    gy = chunks(s["dout"])
    dz = None
    if case["gate"]:
        sig = _sig(z)
        dz = gy * y * sig * (1.0 + z * (1.0 - sig))
        gy = gy * z * sig
    lam = torch.zeros_like(start)
    for i in range(CHUNK - 1, -1, -1):
        lam = decay(i) * (lam + gy[:, :, i, :, None] * cs[i])
    into, carry = torch.empty_like(lam), torch.zeros_like(lam[:, 0])
    for j in range(nc - 1, -1, -1):
        into[:, j] = carry
        carry = torch.exp(total[:, j] * A) * carry + lam[:, j]
    lam, g_in, g_delta = into, torch.empty_like(x), torch.empty_like(x)
    db, dc, da = torch.empty_like(b), torch.empty_like(c), torch.zeros_like(start)
    per_group = lambda v: v.unflatten(2, (-1, group)).sum(3)  # noqa: E731
    for i in range(CHUNK - 1, -1, -1):
        a = decay(i)
        old = a * hs.pop()
        lam = lam + gy[:, :, i, :, None] * cs[i]
        g_in[:, :, i] = (lam * bs[i]).sum(-1)
        g_delta[:, :, i] = (lam * old * A).sum(-1)
        db[:, :, i] = per_group(lam * dx[:, :, i, :, None])
        dc[:, :, i] = per_group(gy[:, :, i, :, None] * (old + dx[:, :, i, :, None] * bs[i]))
        da += lam * old * delta[:, :, i, :, None]
        lam = a * lam
    g_delta += g_in * x
    g_raw = g_delta * _sig(raw) * valid.unflatten(1, (-1, CHUNK))[..., None]
    pack = lambda v: None if v is None else _pack(v.flatten(1, 2), index, valid, t).to(dt)  # noqa: E731
    result["grads"] = {"x": pack(delta * g_in + s["D"] * gy), "dt": pack(g_raw), "B": pack(db), "C": pack(dc),
                       "A": da.sum((0, 1)), "D": (gy * x).sum((0, 1, 2)), "dt_bias": g_raw.sum((0, 1, 2)), "z": pack(dz)}
    return result


def _plain_gated(s):
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    x, z, w = s["x"].float(), s["z"].float(), s["weight"]
    split = lambda v: v.unflatten(1, (case["groups"], -1))  # noqa: E731
    rms = lambda v: (split(v).square().mean(-1, keepdim=True) + EPS).rsqrt()  # noqa: E731
    sig = _sig(z)
    gate = z * sig
    u = x * gate if case["gate_first"] else x
    r = rms(u)
    unit = (split(u) * r).flatten(1)
    out = unit * w if case["gate_first"] else unit * w * gate
    result = {"out": out.to(dt)}
    if case["kind"] == "read":
        return result
    g = s["dout"].float()
    gu = g if case["gate_first"] else g * gate
    dw = (gu * unit).sum(0)
    gu = gu * w
    du = (r * (split(gu) - split(unit) * (split(gu) * split(unit)).mean(-1, keepdim=True))).flatten(1)
    dgate = du * x if case["gate_first"] else g * unit * w
    result["grads"] = {"x": (du * gate if case["gate_first"] else du).to(dt),
                       "z": (dgate * sig * (1.0 + z * (1.0 - sig))).to(dt), "weight": dw}
    return result


def _plain_residual(s):
    case, dt, rt = s["case"], DTYPES[s["case"]["dtype"]], DTYPES[s["case"]["residual"]]
    x, w, scale = s["x"].float(), s["weight"], s["scale"]
    h = s["residual"].float() + (x if scale is None else scale * x)
    r = (h.square().mean(-1, keepdim=True) + EPS).rsqrt()
    unit = h * r
    result = {"out": (unit * w).to(dt), "residual": h.to(rt)}
    if case["kind"] == "read":
        return result
    g = s["dout"].float()
    gw = g * w
    dh = s["dres"].float() + r * (gw - unit * (gw * unit).mean(-1, keepdim=True))
    result["grads"] = {"x": (dh if scale is None else scale * dh).to(dt), "residual": dh.to(rt), "weight": (g * unit).sum(0),
                       "scale": None if scale is None else (dh * x).sum(0)}
    return result


PLAIN = {"conv": _plain_conv, "scan": _plain_scan, "gated": _plain_gated, "residual": _plain_residual}


# ---- 64 bits, from the definitions -----------------------------------------------------------------------------------


def exact(case, seed):
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in _inputs(case, seed).items()}
    return EXACT[case["op"]](case, s)


def _exact_conv(case, s):
    x, w, k, act = s["x"], s["weight"], case["width"], case["kind"] == "act"
    t, d = x.shape
    ends = s["ends"].long()
    episode = torch.searchsorted(ends, torch.arange(t, device="cuda"), right=True)
    starts = ends - torch.tensor(s["lengths"], device="cuda")
    place = torch.arange(t, device="cuda") - starts[episode]

    def back(o):
        """The input o tokens before each token."""
        at = torch.arange(t, device="cuda") - o
        inside = place >= o
        v = x[at.clamp(min=0)] * inside[:, None]
        if "state" in s:
            slot = (k - 1 + place - o).clamp(0, k - 2)
            v = torch.where(inside[:, None], v, s["state"][episode, :, slot])
        return v

    seen = [back(o) for o in range(k)]
    pre = s["bias"] + sum(w[:, k - 1 - o] * seen[o] for o in range(k))
    result = {"out": torch.nn.functional.silu(pre)}
    if case["kind"] != "learn":
        result["state"] = None
        if "state" in s:
            last = ends - 1
            result["state"] = torch.stack([seen[o][last] for o in range(k - 2, -1, -1)], 2)
        return result
    sig = torch.sigmoid(pre)
    dpre = s["dout"] * (sig + pre * sig * (1 - sig))
    dx = dpre * w[:, k - 1]
    for o in range(1, min(k, t)):
        same = (episode[o:] == episode[:t - o])[:, None]
        dx[:t - o] += torch.where(same, dpre[o:], 0.0) * w[:, k - 1 - o]
    result["grads"] = {"x": dx, "weight": torch.stack([(dpre * seen[k - 1 - j]).sum(0) for j in range(k)], 1),
                       "bias": dpre.sum(0)}
    return result


def _exact_scan(case, s):
    t, d = s["x"].shape
    group, learn = d // case["groups"], case["kind"] == "learn"
    x, A, z = s["x"], s["A"], s["z"]
    raw = s["dt"] + s["dt_bias"]
    delta = torch.logaddexp(raw, torch.zeros_like(raw))
    lengths = s["lengths"]
    starts = [0] * len(lengths)
    for i in range(1, len(lengths)):
        starts[i] = starts[i - 1] + lengths[i - 1]
    order = sorted(range(len(lengths)), key=lambda i: -lengths[i])  # the episodes still running come first
    first = torch.tensor([starts[i] for i in order], device="cuda")
    h = s["state"][order] if "state" in s else x.new_zeros(len(lengths), d, case["state"])
    running = [0] * max(lengths)
    for n in lengths:
        running[n - 1] += 1
    for i in range(len(running) - 2, -1, -1):
        running[i] += running[i + 1]
    y, kept = torch.empty_like(x), []
    grow = lambda v, at: v[at].repeat_interleave(group, 1)  # noqa: E731
    for i, n in enumerate(running):
        at = first[:n] + i
        if learn:
            kept.append(h[:n].clone())
        h[:n] = torch.exp(delta[at][..., None] * A) * h[:n] + (delta[at] * x[at])[..., None] * grow(s["B"], at)
        y[at] = torch.einsum("edn,edn->ed", h[:n], grow(s["C"], at))
    y += s["D"] * x
    result = {"out": y * torch.nn.functional.silu(z) if case["gate"] else y}
    if not learn:
        state = torch.empty_like(h)
        state[order] = h
        result["state"] = state if "state" in s else None
        return result
    g = s["dout"]
    dz = None
    if case["gate"]:
        sig = torch.sigmoid(z)
        dz = g * y * (sig + z * sig * (1 - sig))
        g = g * z * sig
    g_x, g_delta = s["D"] * g, torch.zeros_like(x)
    g_b, g_c, g_a = torch.zeros_like(s["B"]), torch.zeros_like(s["C"]), torch.zeros_like(A)
    adj = torch.zeros_like(h)
    for i in range(len(running) - 1, -1, -1):
        n = running[i]
        at = first[:n] + i
        de, xe, b = delta[at][..., None], x[at], grow(s["B"], at)
        a = torch.exp(de * A)
        old = kept.pop()
        lam = adj[:n] + g[at][..., None] * grow(s["C"], at)
        now = a * old + de * xe[..., None] * b
        g_c[at] = (g[at][..., None] * now).unflatten(1, (-1, group)).sum(2)
        g_b[at] = (lam * de * xe[..., None]).unflatten(1, (-1, group)).sum(2)
        to_in = (lam * b).sum(-1)
        g_x[at] += de[..., 0] * to_in
        through = lam * a * old
        g_delta[at] = to_in * xe + (through * A).sum(-1)
        g_a += (through * de).sum(0)
        adj[:n] = a * lam
    g_raw = g_delta * torch.sigmoid(raw)
    result["grads"] = {"x": g_x, "dt": g_raw, "B": g_b, "C": g_c, "A": g_a, "D": (g * x).sum(0), "dt_bias": g_raw.sum(0),
                       "z": dz}
    return result


def _exact_gated(case, s):
    rows, d = s["x"].shape
    shape = (rows, case["groups"], d // case["groups"])
    x, z, w = s["x"].reshape(shape), s["z"].reshape(shape), s["weight"].reshape(shape[1:])
    sig = torch.sigmoid(z)
    gate, slope = z * sig, sig + z * sig * (1 - sig)
    u = x * gate if case["gate_first"] else x
    norm = torch.sqrt((u * u).mean(-1, keepdim=True) + EPS)
    out = w * u / norm * (1 if case["gate_first"] else gate)
    result = {"out": out.reshape(rows, d)}
    if case["kind"] == "learn":
        g = s["dout"].reshape(shape)
        e = g * (1 if case["gate_first"] else gate)  # gradient of w u / norm
        du = w * e / norm - u * (w * e * u).mean(-1, keepdim=True) / norm ** 3
        dx, dz = (du * gate, du * x * slope) if case["gate_first"] else (du, g * w * u / norm * slope)
        result["grads"] = {"x": dx.reshape(rows, d), "z": dz.reshape(rows, d), "weight": (e * u / norm).sum(0).reshape(d)}
    return result


def _exact_residual(case, s):
    x, w = s["x"], s["weight"]
    scale = torch.ones_like(w) if s["scale"] is None else s["scale"]
    h = s["residual"] + scale * x
    norm = torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)
    result = {"out": w * h / norm, "residual": h}
    if case["kind"] == "learn":
        g = s["dout"]
        dh = s["dres"] + w * g / norm - h * (w * g * h).mean(-1, keepdim=True) / norm ** 3
        result["grads"] = {"x": scale * dh, "residual": dh, "weight": (g * h / norm).sum(0),
                           "scale": None if s["scale"] is None else (dh * x).sum(0)}
    return result


EXACT = {"conv": _exact_conv, "scan": _exact_scan, "gated": _exact_gated, "residual": _exact_residual}
