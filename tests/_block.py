"""Inputs and comparisons shared by the tests of state space blocks."""
import numpy as np
import torch

from _delta import bf16, check, ends_of  # noqa: F401

DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
ROUND = {"fp32": lambda x: np.asarray(x, np.float32), "bf16": lambda x: bf16(np.asarray(x, np.float32))}

# Norm-wise bounds, set before the first run.  One rounding to bf16 is at most 2^-8 of a value, 1.7e-3 in the mean
# square over a binade's uniform significands; nothing else is rounded to fewer than 24 bits, so 2.5e-3 leaves room for
# unlucky significands of few values.
ROUNDED = {"fp32": 0.0, "bf16": 2.5e-3}
# Rows that sum at most a few dozen fp32 terms, each off by a few 2^-24, and gates from expf and a fast division, 2^-22.
ROW = 2e-6
# The scan: a decay exp2(delta A2) is off by 2^-21 at most (2^-22 of ex2.approx, rounded product and A2), and a state
# remembers up to about 30 tokens of it here (delta |A| above 1/30 on average): 30 x 2^-21 = 1.4e-5 were all of them of
# one sign and the largest.
SCAN = 1.5e-5
# Sums over tokens of products of either sign: their own terms cancel by up to sqrt(tokens) against the norm of the
# terms; held against the whole gradient's norm.
SUM = 3e-5


def dev(x, dtype="fp32"):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda().to(DT[dtype])


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def junk(*shape, dtype="fp32"):
    """Every output starts as NaN: what is not written shows."""
    return torch.full(shape, float("nan"), device="cuda", dtype=DT[dtype])


def strided(parts, pad=8):
    """The same values as slices of one wide buffer (and the buffer)."""
    t = parts[0].shape[0]
    wide = torch.cat([p.reshape(t, -1) for p in parts] + [torch.zeros(t, pad, device="cuda", dtype=parts[0].dtype)], 1)
    out, at = [], 0
    for p in parts:
        n = p[0].numel() if t else int(np.prod(p.shape[1:]))
        out.append(wide[:, at:at + n].unflatten(1, p.shape[1:]) if p.dim() > 2 else wide[:, at:at + n])
        at += n
    return out, wide


def conv_inputs(lengths, channels, width, seed, dtype):
    r, rnd = np.random.default_rng(seed), ROUND[dtype]
    t, n = int(np.sum(lengths)), len(lengths)
    state = (n, channels, width - 1)
    return dict(x=rnd(r.standard_normal((t, channels))), w=np.float32(r.standard_normal((channels, width)) / width ** 0.5),
                bias=np.float32(r.standard_normal(channels)), dout=rnd(r.standard_normal((t, channels))),
                init=rnd(r.standard_normal(state)), d_final=rnd(r.standard_normal(state)))


def scan_inputs(lengths, channels, n, groups, seed, dtype, softplus=True):
    r, rnd = np.random.default_rng(seed), ROUND[dtype]
    t, e = int(np.sum(lengths)), len(lengths)
    f = np.float32
    # delta about 0.02 to 0.5, |A| from 0.5 on
    dt = r.standard_normal((t, channels)) - 2.0 if softplus else r.uniform(0.02, 0.5, (t, channels))
    return dict(x=rnd(r.standard_normal((t, channels))), dt=rnd(dt), A=f(-0.5 * np.exp(r.uniform(0, 3, (channels, n)))),
                B=rnd(r.standard_normal((t, groups, n))), C=rnd(r.standard_normal((t, groups, n))),
                D=f(r.standard_normal(channels)), z=rnd(r.standard_normal((t, channels))),
                dt_bias=f(0.3 * r.standard_normal(channels)), dout=rnd(r.standard_normal((t, channels))),
                init=f(r.standard_normal((e, channels, n))), d_final=f(r.standard_normal((e, channels, n))))
