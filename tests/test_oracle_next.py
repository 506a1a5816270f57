"""The 64-bit oracle of norm_quantize, the block product and sampling against
closed forms and brute force."""

import math

import numpy as np
import pytest

from oracle import codecs, next_token as nt

GRID = np.array([v for v in codecs.e4m3_decode(np.arange(127, dtype=np.uint8))])


@pytest.mark.parametrize("most,e", [(448.0, 0), (np.nextafter(448.0, 500), 1), (224.0, -1), (1.75, -8), (1.0, -8), (0.875, -9),
                                    (0.0, -127), (1e-45, -127), (3e38, 120), (448 * 2.0 ** -127, -127), (500 * 2.0 ** -127, -126)])
def test_exponent(most, e):
    assert nt.exponent(most) == e


def test_block_codes_are_nearest():
    g = np.random.default_rng(0)
    h = g.standard_normal((3, 256)) * np.exp(g.standard_normal((3, 1)) * 5)
    h[1, 128:] = 0
    codes, scales = nt.quantize_rows(h, nt.FP8_BLOCK)
    assert scales.shape == (3, 4) and not scales[:, 2:].any()
    got = nt.values(codes, scales, 1)
    for i in range(3):
        for j in range(256):
            step = 2.0 ** (int(scales[i, j // 128]) - 127)
            assert abs(got[i, j] - h[i, j]) <= np.abs(np.abs(h[i, j]) - GRID * step).min() * (1 + 1e-12)
    # the largest of a block uses the upper half of the range
    top = np.abs(codecs.e4m3_decode(codes)).reshape(3, 2, 128).max(-1)
    assert ((top > 216) | (np.abs(h).reshape(3, 2, 128).max(-1) == 0)).all()


@pytest.mark.parametrize("fmt", [nt.FP8_ROW, nt.INT8_ROW])
def test_row_codes(fmt):
    g = np.random.default_rng(1)
    h = g.standard_normal((4, 64))
    h[2] = 0
    h[3, 5] = np.inf
    codes, scales = nt.quantize_rows(h, fmt)
    assert scales[2] == 0 and not codes[2].any() and np.isnan(scales[3]) and not codes[3].any()
    vals = codes.view(np.int8).astype(float) if fmt == nt.INT8_ROW else codecs.e4m3_decode(codes)
    most = 127 if fmt == nt.INT8_ROW else 448
    assert (np.abs(vals[:2]).max(1) == most).all()
    err = np.abs(vals[:2] * scales[:2, None] - h[:2])
    half = 0.5 * scales[:2, None] if fmt == nt.INT8_ROW else np.maximum(2.0 ** -4 * np.abs(h[:2]), 2.0 ** -10 * scales[:2, None])
    assert (err <= half * (1 + 1e-6)).all()


def test_norms():
    x = np.array([[3.0, -4.0]])
    assert np.allclose(nt.normed(x, nt.RMS, None, None, 0.0), x / math.sqrt(12.5))
    assert np.allclose(nt.normed(x, nt.LAYER, np.array([2.0, 1.0]), np.array([0.0, 5.0]), 0.0), [[2.0, 4.0]])
    assert (nt.normed(x, nt.NONE, np.array([2.0, 1.0]), None, 0.0) == [[6.0, -4.0]]).all()


def test_product_is_the_sum_over_blocks():
    g = np.random.default_rng(2)
    xq, sx = nt.quantize_rows(g.standard_normal((3, 384)), nt.FP8_BLOCK)
    wq, sw = nt.quantize_weight(g.standard_normal((130, 384)))
    assert sw.shape == (2, 4)
    y, _ = nt.product(xq, sx, wq, sw)
    m, n = 2, 129
    want = sum(2.0 ** (int(sx[m, b]) + int(sw[1, b]) - 254) *
               float(codecs.e4m3_decode(xq[m, 128 * b:128 * b + 128]) @ codecs.e4m3_decode(wq[n, 128 * b:128 * b + 128]))
               for b in range(3))
    assert abs(y[m, n] - want) < 1e-9
    sx[m, 1] = 255
    assert np.isnan(nt.product(xq, sx, wq, sw)[0][m]).all()


def test_sampling_closed_forms():
    z = np.log(np.array([1.0, 4.0, 2.0, 4.0, 1.0]))
    at = lambda **kw: nt.kept(z, kw.get("T", 1.0), kw.get("k", 0), kw.get("p", 1.0), kw.get("m", 0.0))[0].tolist()  # noqa: E731
    assert at() == [0, 1, 2, 3, 4]
    assert at(k=1) == [1] and at(k=2) == [1, 3] and at(k=4) == [0, 1, 2, 3]     # equal ones by rising index
    # masses in order: 4 4 2 1 1 of 12
    assert at(p=4 / 12 - 1e-6) == [1] and at(p=0.5) == [1, 3] and at(p=0.8) == [1, 2, 3] and at(p=0.0) == [1]
    assert at(p=0.5, k=1) == [1]
    assert at(m=0.4) == [1, 2, 3] and at(m=2.0) == [1, 3] and at(T=0.0) == [1]
    # top_p is of what top_k left: 4 of 8
    assert at(k=2, p=0.5) == [1] and at(k=2, p=0.51) == [1, 3]
    # draws by index: 1 4 2 4 1 of 12
    for u, want in ((0.0, 0), (0.083, 0), (0.0834, 1), (0.41, 1), (0.42, 2), (0.9, 3), (0.9999, 4), (1.0, 4), (7.0, 4), (math.nan, 0)):
        assert nt.sample(z, u=u)[0] == want, u
    assert abs(nt.sample(z, u=0.5)[1] - math.log(2 / 12)) < 1e-12
    assert nt.sample(np.full(4, -np.inf)) == (-1, -math.inf)
    assert nt.sample(np.array([np.nan, 0.0, -np.inf]), u=0.9)[0] == 1
    assert nt.sample(np.array([5.0, np.inf, 2.0, np.inf]), u=0.6)[0] == 3


def test_sampling_frequencies():
    g = np.random.default_rng(3)
    z = g.standard_normal(12)
    at, w = nt.kept(z, 0.7, 8, 0.9, 0.05)
    n = 4000
    got = np.bincount([nt.sample(z, 0.7, 8, 0.9, 0.05, (i + 0.5) / n)[0] for i in range(n)], minlength=12) / n
    want = np.zeros(12)
    want[at] = w[at] / w[at].sum()
    # evenly spaced numbers: each count is off by at most two of them
    assert np.abs(got - want).max() <= 2 / n
