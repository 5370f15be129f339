"""The fp64 gated delta rule: what the recurrence must do, and its adjoint against differences."""
import numpy as np
import pytest

from _delta import ends_of, inputs
from oracle import delta


def _args(d):
    return [np.asarray(d[x], np.float64) for x in ("q", "k", "v", "g", "beta")]


def test_a_unit_key_with_full_strength_reads_back_its_value():
    k = np.zeros((1, 1, 4))
    k[0, 0, 2] = 1.0
    v = np.arange(3.0).reshape(1, 1, 3)
    out, final = delta.forward(k, k, v, np.zeros((1, 1)), np.ones((1, 1)), [1], 1.0,
                               init=np.ones((1, 1, 3, 4)))
    np.testing.assert_allclose(out[0, 0], v[0, 0])
    np.testing.assert_allclose(final[0, 0, :, 2], v[0, 0])       # the key's column is replaced
    np.testing.assert_allclose(final[0, 0, :, [0, 1, 3]], 1.0)   # the others stay


def test_no_strength_only_decays_and_minus_infinity_forgets():
    d = inputs([5], 1, 2, 4, 3, 0)
    a = _args(d)
    a[4][:] = 0.0
    _, final = delta.forward(*a, [5], 1.0, init=d["init"])
    np.testing.assert_allclose(final[0], d["init"][0] * np.exp(a[3].sum(0))[:, None, None])
    a = _args(d)
    a[3][2] = -np.inf
    _, full = delta.forward(*a, [5], 1.0, init=d["init"])
    _, late = delta.forward(*[x[2:] for x in a], [3], 1.0)
    np.testing.assert_allclose(full, late)


def test_episodes_are_apart_and_heads_share_keys():
    lengths = [3, 0, 1, 4]
    d = inputs(lengths, 2, 4, 4, 3, 1)
    out, final = delta.forward(*_args(d), ends_of(lengths), 0.5, init=d["init"])
    lo = 0
    for e, n in enumerate(lengths):
        o, f = delta.forward(*[x[lo:lo + n] for x in _args(d)], [n], 0.5, init=d["init"][e:e + 1])
        np.testing.assert_allclose(out[lo:lo + n], o)
        np.testing.assert_allclose(final[e], f[0])
        lo += n
    np.testing.assert_array_equal(final[1], d["init"][1])
    q, k, v, g, b = _args(d)
    o, _ = delta.forward(q[:, 1:], k[:, 1:], v[:, 3:], g[:, 3:], b[:, 3:], ends_of(lengths), 0.5,
                         init=d["init"][:, 3:])
    np.testing.assert_allclose(o[:, 0], out[:, 3])


@pytest.mark.parametrize("k_heads,v_heads", [(1, 1), (1, 3), (2, 4)])
def test_adjoint_against_differences(k_heads, v_heads):
    lengths = [4, 1, 0, 3]
    d = inputs(lengths, k_heads, v_heads, 3, 2, 7)
    ends, scale = ends_of(lengths), 0.7
    names = ("q", "k", "v", "g", "beta", "init")
    base = {n: np.asarray(d[n], np.float64) for n in names}

    def loss(x):
        out, final = delta.forward(x["q"], x["k"], x["v"], x["g"], x["beta"], ends, scale, init=x["init"])
        return (out * d["dout"]).sum() + (final * d["d_final"]).sum()

    grads = delta.backward(*[base[n] for n in names[:5]], ends, scale, d["dout"], init=base["init"],
                           d_final=d["d_final"])
    h = 1e-5
    for name, grad in zip(names, grads):
        for at in np.ndindex(*base[name].shape):
            hi, lo = ({n: x.copy() for n, x in base.items()} for _ in range(2))
            hi[name][at] += h
            lo[name][at] -= h
            # central differences: O(h^2) truncation plus 2^-53 |loss| / h rounding
            assert abs((loss(hi) - loss(lo)) / (2 * h) - grad[at]) < 1e-7, (name, at)
