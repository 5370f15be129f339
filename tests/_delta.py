"""Inputs and comparisons shared by the tests of the gated delta rule."""
import numpy as np

# Half the spacing of the token types over a binade's top: what rounding once may cost in the norm of many values
# (1.7e-3 in the mean square for bf16; a single value is off by up to twice this, so single values are compared
# with the reference rounded to the type).
U = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -9}

# Norm-wise bounds, set before the first run.  fp32: operands carry at least
# 22 significand bits (2^-23 relative to their tile's largest element) through
# at most about ten products, sums are fp32 (2^-24 each, up to 192 terms), and
# the gradient of the log decay is a suffix sum of differences: 1e-5 leaves
# room for that cancellation.  bf16 tokens: the output's own rounding (at most
# 2^-8, 1.7e-3 in the mean square over a binade's uniform significands) plus
# operands of 11 bits (2^-12 each, about ten of them).
BOUND = {"fp32": 1e-5, "bf16": 4e-3}
STATE_BOUND = 1e-5        # states are fp32 whatever the tokens are


def bf16(x):
    """Nearest bfloat16 of fp32 values, as fp32."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32)
    r = ((b >> 16) & 1) + 0x7FFF
    return ((b + r) & 0xFFFF0000).view(np.float32)


def ends_of(lengths):
    return np.cumsum(lengths).astype(np.int32)


def inputs(lengths, k_heads, v_heads, k_dim, v_dim, seed, decay=1.0, rnd=lambda x: x):
    """q, k (unit rows, positively correlated), v, g <= 0, beta in (0, 1), dout, and states."""
    r = np.random.default_rng(seed)
    t = int(np.sum(lengths))

    def unit(*s):
        x = r.standard_normal(s) + 0.3
        return x / np.maximum(np.linalg.norm(x, axis=-1, keepdims=True), 1e-6)

    f = lambda x: rnd(np.asarray(x, np.float32))
    d = dict(q=f(unit(t, k_heads, k_dim)), k=f(unit(t, k_heads, k_dim)), v=f(r.standard_normal((t, v_heads, v_dim))),
             g=f(-decay * r.exponential(0.1, (t, v_heads))), beta=f(1 / (1 + np.exp(-r.standard_normal((t, v_heads))))),
             dout=f(r.standard_normal((t, v_heads, v_dim))))
    shape = (len(lengths), v_heads, v_dim, k_dim)
    d["init"] = (0.3 * r.standard_normal(shape)).astype(np.float32)
    d["d_final"] = (0.3 * r.standard_normal(shape)).astype(np.float32)
    return d


def off(got, want):
    """|got - want| / |want| in the 2-norm (0 / 0 = 0)."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    n = np.linalg.norm(want)
    d = np.linalg.norm(got - want)
    return 0.0 if d == 0 else (np.inf if n == 0 else d / n)


def check(got, want, bound, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, f"{what}: shape {got.shape}, want {want.shape}"
    assert np.isfinite(got).all(), f"{what}: {np.count_nonzero(~np.isfinite(got))} non-finite values"
    rel = off(got, want)
    assert rel <= bound, f"{what}: off by {rel:.3g} in the norm (bound {bound:.3g})"
    if want.size:      # no single element far off: 40 bounds of its own size or of the root mean square
        rms = np.linalg.norm(want) / np.sqrt(want.size)
        worst = np.max(np.abs(got - want) / np.maximum(np.abs(want), max(rms, 1e-300)))
        assert worst <= 40 * bound, f"{what}: an element off by {worst:.3g} (bound {40 * bound:.3g})"
