"""The 64-bit oracle of the time-mix operators: gradients against central
differences, and forms that have closed values.

Differences with step h of a smooth function have an error of h^2 f'''/6 plus
roundoff 2^-52 |f| / h; at h = 1e-5 and values of order 1e2 both stay below
1e-7 of the gradient's scale, so 1e-6 of it is the bound."""

import math

import numpy as np
import pytest

from oracle import mix

LENS = [3, 0, 1, 4]
T = sum(LENS)


def _directional(f, x, d, h=1e-5):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


def _check(loss, args, grads, seed):
    g = np.random.default_rng(seed)
    for name, x in args.items():
        d = g.standard_normal(x.shape)
        want = _directional(lambda z: loss(dict(args, **{name: z})), x, d)
        got = float((grads[name] * d).sum())
        scale = float(np.abs(grads[name] * d).sum()) + 1e-12
        assert abs(got - want) <= 1e-6 * scale, (name, got, want)


@pytest.mark.parametrize("heads", [1, 2])
def test_time_mix_gradient(heads):
    g = np.random.default_rng(heads)
    c = 64 * heads
    args = {q: g.standard_normal((T, c)) * (0.2 if q in "ab" else 1.0) for q in "rwkvab"}
    args["state"] = g.standard_normal((len(LENS), heads, 64, 64))
    dy, ds = g.standard_normal((T, c)), g.standard_normal((len(LENS), heads, 64, 64))

    def loss(q):
        y, S = mix.time_mix(*(q[z] for z in "rwkvab"), LENS, q["state"])
        return float((y * dy).sum() + (S * ds).sum())

    got = mix.time_mix_backward(*(args[z] for z in "rwkvab"), LENS, args["state"], dy, ds)
    _check(loss, args, {**{z: got["d" + z] for z in "rwkvab"}, "state": got["dstate"]}, 10 + heads)


def test_time_mix_closed_forms():
    g = np.random.default_rng(3)
    k, v, r = (g.standard_normal((5, 64)) for _ in range(3))
    zero = np.zeros((5, 64))
    # a decay of sigmoid(0) = 1/2 everywhere and no removal: a decayed sum of outer products
    y, S = mix.time_mix(r, zero, k, v, zero, zero, [5])
    w = math.exp(-0.5 * math.exp(-0.5))
    want = sum(w ** (4 - t) * np.outer(v[t], k[t]) for t in range(5))
    assert np.allclose(S[0, 0], want, rtol=1e-13, atol=1e-13)
    assert np.allclose(y[4], want @ r[4], rtol=1e-12, atol=1e-12)
    # a = -kappa, b = kappa with a unit kappa and no decay: the state forgets kappa's direction
    kap = g.standard_normal((1, 64))
    kap /= np.linalg.norm(kap)
    S0 = g.standard_normal((1, 1, 64, 64))
    _, S = mix.time_mix(kap, np.full((1, 64), -800.0), np.zeros((1, 64)), np.zeros((1, 64)), -kap, kap, [1], S0)
    assert np.allclose(S[0, 0] @ kap[0], 0, atol=1e-13)
    # an empty sequence keeps its state
    y, S = mix.time_mix(*(np.zeros((0, 64)),) * 6, [0], S0)
    assert y.shape == (0, 64) and np.array_equal(S, S0)


def test_shift_norm_gradient():
    g = np.random.default_rng(4)
    c, m = 24, 3
    args = {"x": g.standard_normal((T, c)), "gamma": g.standard_normal(c), "beta": g.standard_normal(c),
            "mu": g.random((m, c)), "shift": g.standard_normal((len(LENS), c))}
    dout, dx, dsh = g.standard_normal((m, T, c)), g.standard_normal((T, c)), g.standard_normal((len(LENS), c))

    def loss(q):
        x, out, last = mix.shift_norm(q["x"], None, 0.0, LENS, q["gamma"], q["beta"], 1e-5, q["mu"], q["shift"])
        return float((out * dout).sum() + (x * dx).sum() + (last * dsh).sum())

    got = mix.shift_norm_backward(args["x"], LENS, args["gamma"], args["beta"], 1e-5, args["mu"], args["shift"], dout, dx, dsh)
    _check(loss, args, {"x": got["dx"], "gamma": got["dgamma"], "beta": got["dbeta"], "mu": got["dmu"],
                        "shift": got["dshift_in"]}, 5)


def test_head_gate_gradient():
    g = np.random.default_rng(6)
    c = 128
    args = {q: g.standard_normal((T, c)) for q in "yrkvg"}
    args.update({q: g.standard_normal(c) for q in ("gamma", "beta", "u")})
    dout = g.standard_normal((T, c))

    def loss(q):
        return float((mix.head_gate(*(q[z] for z in "yrkvg"), q["gamma"], q["beta"], 64e-5, q["u"]) * dout).sum())

    got = mix.head_gate_backward(*(args[z] for z in "yrkvg"), args["gamma"], args["beta"], 64e-5, args["u"], dout)
    names = {z: "d" + z for z in ("y", "r", "k", "v", "g", "gamma", "beta", "u")}
    _check(loss, args, {q: got[n] for q, n in names.items()}, 7)
