"""64-bit oracle of the operators between an RWKV-7 layer's projections: the
shifted norm and its mixtures, the state recurrence, the head norm and gate,
and their gradients, each written token by token from its definition.

Arrays are numpy float64; rows are [tokens][width], states
[sequence][head][64 channels of v][64 channels of k], `lens` the sequences'
lengths.  Gradients are the formulas' own, checked against differences in
tests/test_oracle_mix.py.
"""

import math

import numpy as np

HEAD = 64
DECAY = math.exp(-0.5)


def sigmoid(x):
    return 0.5 * (1.0 + np.tanh(0.5 * x))


def _heads(x):
    return np.asarray(x, dtype=np.float64).reshape(x.shape[0], x.shape[1] // HEAD, HEAD)


def time_mix(r, w, k, v, a, b, lens, states=None, keep=None):
    """(y [tokens][width], states after each sequence).  keep: a list that gets
    the state before every token."""
    r, w, k, v, a, b = (_heads(x) for x in (r, w, k, v, a, b))
    n, heads = len(lens), r.shape[1]
    decay = np.exp(-DECAY * sigmoid(w))
    S = np.zeros((n, heads, HEAD, HEAD)) if states is None else np.array(states, dtype=np.float64)
    y = np.zeros_like(r)
    t = 0
    for i, m in enumerate(lens):
        for _ in range(m):
            if keep is not None:
                keep.append(S[i].copy())
            u = np.einsum("hij,hj->hi", S[i], a[t])
            S[i] = S[i] * decay[t][:, None, :] + u[:, :, None] * b[t][:, None, :] + v[t][:, :, None] * k[t][:, None, :]
            y[t] = np.einsum("hij,hj->hi", S[i], r[t])
            t += 1
    return y.reshape(t, -1) if t else y.reshape(0, heads * HEAD), S


def time_mix_backward(r, w, k, v, a, b, lens, states, dy, dstates=None):
    """The gradients of sum(y dy) + sum(states' dstates): a dict of dr, dw, dk,
    dv, da, db [tokens][width] and dstate."""
    before = []
    _, after = time_mix(r, w, k, v, a, b, lens, states, keep=before)
    r, w, k, v, a, b, dy = (_heads(x) for x in (r, w, k, v, a, b, dy))
    sg = sigmoid(w)
    decay = np.exp(-DECAY * sg)
    D = np.zeros_like(after) if dstates is None else np.array(dstates, dtype=np.float64)
    g = {q: np.zeros_like(r) for q in ("dr", "dw", "dk", "dv", "da", "db")}
    ends = np.cumsum(lens)
    for i, m in enumerate(lens):
        S = after[i]
        for t in range(ends[i] - 1, ends[i] - m - 1, -1):
            g["dr"][t] = np.einsum("hij,hi->hj", S, dy[t])
            D[i] += dy[t][:, :, None] * r[t][:, None, :]
            S = before[t]
            u = np.einsum("hij,hj->hi", S, a[t])
            du = np.einsum("hij,hj->hi", D[i], b[t])
            g["dv"][t] = np.einsum("hij,hj->hi", D[i], k[t])
            g["dk"][t] = np.einsum("hij,hi->hj", D[i], v[t])
            g["db"][t] = np.einsum("hij,hi->hj", D[i], u)
            g["da"][t] = np.einsum("hij,hi->hj", S, du)
            dw = (D[i] * S).sum(1)
            g["dw"][t] = dw * decay[t] * -DECAY * sg[t] * (1.0 - sg[t])
            D[i] = D[i] * decay[t][:, None, :] + du[:, :, None] * a[t][:, None, :]
    out = {q: x.reshape(x.shape[0], -1) for q, x in g.items()}
    out["dstate"] = D
    return out


def _normed(x, eps):
    mid = x - x.mean(-1, keepdims=True)
    rstd = 1.0 / np.sqrt((mid * mid).mean(-1, keepdims=True) + eps)
    return mid * rstd, rstd


def _norm_back(dn, n, rstd):
    return (dn - dn.mean(-1, keepdims=True) - n * (dn * n).mean(-1, keepdims=True)) * rstd


def _before(h, lens, shift):
    """The row before each row, and the index of each sequence's first row."""
    prev = np.zeros_like(h)
    prev[1:] = h[:-1]
    t = 0
    for i, m in enumerate(lens):
        if m:
            prev[t] = 0.0 if shift is None else shift[i]
        t += m
    return prev


def shift_norm(x, delta, alpha, lens, gamma, beta, eps, mu, shift=None):
    """(x', out [nmix][tokens][width], shift after each sequence)."""
    full = np.asarray(x, dtype=np.float64) + (0.0 if delta is None else alpha * np.asarray(delta, dtype=np.float64))
    h = _normed(full, eps)[0] * gamma + beta
    prev = _before(h, lens, shift)
    out = np.stack([h + (prev - h) * m for m in mu])
    last = np.zeros((len(lens), h.shape[1])) if shift is None else np.array(shift, dtype=np.float64)
    t = 0
    for i, m in enumerate(lens):
        t += m
        if m:
            last[i] = h[t - 1]
    return full, out, last


def shift_norm_backward(x, lens, gamma, beta, eps, mu, shift, dout, dx_out=None, dshift_out=None):
    """Gradients of sum(out dout) + sum(x dx_out) + sum(shift' dshift_out)."""
    x = np.asarray(x, dtype=np.float64)
    n, rstd = _normed(x, eps)
    h = n * gamma + beta
    prev = _before(h, lens, shift)
    dprev = (dout * mu[:, None, :]).sum(0)
    dh = dout.sum(0) - dprev
    dmu = (dout * (prev - h)).sum(1)
    dshift = np.zeros((len(lens), x.shape[1]))
    t = 0
    for i, m in enumerate(lens):
        if m:
            dshift[i] = dprev[t]
            dh[t:t + m - 1] += dprev[t + 1:t + m]
            if dshift_out is not None:
                dh[t + m - 1] += dshift_out[i]
        elif dshift_out is not None:
            dshift[i] = dshift_out[i]
        t += m
    dx = _norm_back(dh * gamma, n, rstd)
    if dx_out is not None:
        dx = dx + dx_out
    return {"dx": dx, "dgamma": (dh * n).sum(0), "dbeta": dh.sum(0), "dmu": dmu, "dshift_in": dshift}


def head_gate(y, r, k, v, g, gamma, beta, eps, u):
    y, r, k, v, g = (_heads(x) for x in (y, r, k, v, g))
    gamma, beta, u = (np.asarray(x, dtype=np.float64).reshape(-1, HEAD) for x in (gamma, beta, u))
    n = _normed(y, eps)[0]
    out = (n * gamma + beta + (r * k * u).sum(-1, keepdims=True) * v) * g
    return out.reshape(out.shape[0], -1)


def head_gate_backward(y, r, k, v, g, gamma, beta, eps, u, dout):
    y, r, k, v, g, dout = (_heads(x) for x in (y, r, k, v, g, dout))
    gamma, beta, u = (np.asarray(x, dtype=np.float64).reshape(-1, HEAD) for x in (gamma, beta, u))
    n, rstd = _normed(y, eps)
    bonus = (r * k * u).sum(-1, keepdims=True)
    dz = dout * g
    db = (dz * v).sum(-1, keepdims=True)
    out = {"dy": _norm_back(dz * gamma, n, rstd), "dr": db * k * u, "dk": db * r * u, "dv": dz * bonus,
           "dg": dout * (n * gamma + beta + bonus * v)}
    out = {q: x.reshape(x.shape[0], -1) for q, x in out.items()}
    out.update(dgamma=(dz * n).sum(0).reshape(-1), dbeta=dz.sum(0).reshape(-1), du=(db * r * k).sum(0).reshape(-1))
    return out
