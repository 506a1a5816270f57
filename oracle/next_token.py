"""64-bit oracle of what follows a model's last layer: the norm that leaves
8-bit rows, the fp8 product with a power of two per block of 128, and sampling,
each written from its definition.  Arrays are numpy; e4m3 codes are uint8.
"""

import math

import numpy as np

from . import codecs

BLOCK = 128
NONE, RMS, LAYER = range(3)
FP8_ROW, INT8_ROW, FP8_BLOCK = 4, 5, 11    # the library's format numbers


def scale_row(k):
    """Bytes of one row of block scales."""
    return 4 * -(-k // (4 * BLOCK))


def exponent(most):
    """The smallest e in -127..127 with most <= 448 * 2^e."""
    if most <= 0:
        return -127
    e = math.frexp(most / 448.0)[1] - 1
    while most > math.ldexp(448.0, e):
        e += 1
    while most <= math.ldexp(448.0, e - 1):
        e -= 1
    return min(max(e, -127), 127)


def normed(x, kind, gamma, beta, eps):
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(all="ignore"):
        if kind == RMS:
            x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        elif kind == LAYER:
            x = x - x.mean(-1, keepdims=True)
            x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        if gamma is not None:
            x = x * gamma
        if beta is not None:
            x = x + beta
    return x


def quantize_rows(h, fmt):
    """(codes uint8 [rows][width], scales): fp32 [rows] or E8M0 bytes [rows][scale_row]."""
    rows, width = h.shape
    codes = np.zeros((rows, width), dtype=np.uint8)
    group = BLOCK if fmt == FP8_BLOCK else width
    scales = np.zeros((rows, scale_row(width)), dtype=np.uint8) if fmt == FP8_BLOCK else np.zeros(rows, dtype=np.float32)
    for i in range(rows):
        for b in range(width // group):
            part = h[i, b * group:(b + 1) * group]
            at = (i, slice(b * group, (b + 1) * group))
            if not np.isfinite(part).all():
                if fmt == FP8_BLOCK:
                    scales[i, b] = 255
                else:
                    scales[i] = np.nan
                continue
            most = float(np.abs(part).max())
            if fmt == FP8_BLOCK:
                e = exponent(most)
                scales[i, b] = e + 127
                codes[at] = codecs.e4m3_encode(part * math.ldexp(1.0, -e))
            else:
                s = np.float32(most / (127.0 if fmt == INT8_ROW else 448.0))
                scales[i] = s
                if s > 0:
                    q = part / float(s)
                    codes[at] = np.clip(np.rint(q), -127, 127).astype(np.int8).view(np.uint8) if fmt == INT8_ROW \
                        else codecs.e4m3_encode(q)
    return codes, scales


def quantize_weight(w):
    """(codes [n][k], scale bytes [ceil(n/128)][scale_row(k)]) of RQ_FP8_E4M3_B128."""
    n, k = w.shape
    codes = np.zeros((n, k), dtype=np.uint8)
    scales = np.zeros((-(-n // BLOCK), scale_row(k)), dtype=np.uint8)
    for i in range(scales.shape[0]):
        for b in range(k // BLOCK):
            at = (slice(i * BLOCK, (i + 1) * BLOCK), slice(b * BLOCK, (b + 1) * BLOCK))
            part = w[at].astype(np.float64)
            e = exponent(float(np.abs(part).max()))
            scales[i, b] = e + 127
            codes[at] = codecs.e4m3_encode(part * math.ldexp(1.0, -e))
    return codes, scales


def values(codes, scales, rows_per):
    """What codes [n][k] with block scales stand for."""
    n, k = codes.shape
    e = scales[:, :k // BLOCK].astype(np.float64)
    step = np.where(e == 255, np.nan, np.exp2(e - 127)).repeat(BLOCK, 1).repeat(rows_per, 0)[:n]
    return codecs.e4m3_decode(codes) * step


def product(xq, sx, wq, sw):
    """(y [m][n], sum |x w|)."""
    x, w = values(xq, sx, 1), values(wq, sw, BLOCK)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def kept(z, temperature, top_k, top_p, min_p):
    """Indices that stay after the filters, rising, and the weights of all."""
    z = np.asarray(z, dtype=np.float64)
    z = np.where(np.isnan(z), -np.inf, z)
    top = z.max()
    if not top > -np.inf:
        return np.zeros(0, dtype=np.int64), np.zeros_like(z)
    if not temperature > 0:
        return np.array([int(np.argmax(z == top))]), (z == top).astype(np.float64)
    if np.isposinf(top):
        w = (z == top).astype(np.float64)
    else:
        with np.errstate(all="ignore"):
            w = np.where(z == -np.inf, 0.0, np.exp((z - top) / float(temperature)))
    order = np.argsort(-z, kind="stable")
    n = len(order)
    if top_k > 0:
        n = min(n, int(top_k))
    if top_p < 1:
        mass = np.cumsum(w[order[:n]])
        n = 1 + int(np.sum(mass[:-1] < float(top_p) * mass[-1]))
    order = order[:n]
    if min_p > 0:
        order = order[w[order] >= min(float(min_p), 1.0)]
    order = order[w[order] > 0]
    return np.sort(order), w


def sample(z, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, u=0.0):
    """(token, logprob) of one row; parameters as the fp32 values that the call gets."""
    at, w = kept(z, temperature, top_k, top_p, min_p)
    if not len(at):
        return -1, -math.inf
    u = 0.0 if not u > 0 else min(float(u), 1.0 - 2.0 ** -24)
    mass = np.cumsum(w[at])
    j = min(int(np.searchsorted(mass, u * mass[-1], side="right")), len(at) - 1)
    return int(at[j]), math.log(w[at[j]] / mass[-1])
