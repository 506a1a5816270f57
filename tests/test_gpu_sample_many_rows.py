"""Draws for more than 256 rows, whose workgroups have half the waves and twice the
turns, against the 64-bit oracle: tokens equal, log-probabilities as in
test_gpu_sample.  Every row is drawn, some thirty of them are checked, the first and
the last among them."""

import math

import numpy as np
import pytest
import torch

from oracle import next_token as nt
from test_gpu_sample import FILTERS, TYPES, f32, logits_of, run

pytestmark = pytest.mark.gpu


def check_some(logits, vocab, T=None, k=None, p=None, m=None, u=0.0, seed=0):
    rows = logits.shape[0]
    got, lp = run(logits, vocab, T, k, p, m, u)
    some = sorted({0, 1, 255, 256, rows - 1} | set(np.random.default_rng(seed).integers(0, rows, 27).tolist()))
    z = logits[some, :vocab].double().cpu().numpy()

    def at(v, i, default):
        return default if v is None else f32(v if np.isscalar(v) else v[i])
    for i, row in zip(some, z):
        want, wlp = nt.sample(row, at(T, i, 1.0), at(k, i, 0), at(p, i, 1.0), at(m, i, 0.0), at(u, i, 0.0))
        assert got[i] == want, (i, got[i], want, lp[i], wlp)
        assert abs(lp[i] - wlp) <= 1e-6 + 2.0 ** -23 * abs(wlp), (i, lp[i], wlp)


@pytest.mark.parametrize("filters", FILTERS)
@pytest.mark.parametrize("dtype,rows,vocab", [("f16", 257, 50277), ("bf16", 300, 20011), ("f32", 261, 65536), ("f16", 509, 4097),
                                              ("f32", 270, 131072)])
def test_draws(dtype, rows, vocab, filters):
    g = np.random.default_rng(rows)
    check_some(logits_of(vocab + 1, rows, vocab, dtype), vocab, u=list(g.random(rows)), **FILTERS[filters])


@pytest.mark.parametrize("dtype", TYPES)
def test_parameters_of_their_own(dtype):
    rows, vocab = 400, 30011
    g = np.random.default_rng(8)
    check_some(logits_of(2, rows, vocab, dtype), vocab, T=list(np.where(g.random(rows) < 0.1, 0, 0.3 + 1.5 * g.random(rows))),
               k=[int(v) for v in np.where(g.random(rows) < 0.5, np.exp(g.random(rows) * 9).astype(int), 0)],
               p=list(np.where(g.random(rows) < 0.5, g.random(rows), 1.0)), m=list(np.where(g.random(rows) < 0.5, 0.2 * g.random(rows), 0)),
               u=list(g.random(rows)))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("levels", [1, 2, 5, 40, 3000])
def test_ties(dtype, levels):
    """More than a list's 512 equal logits on either side of a border, over several turns."""
    rows, vocab = 260, 33000
    g = np.random.default_rng(levels)
    z = g.integers(0, levels, (rows, vocab)).astype(np.float64) * (10.0 / levels)
    z[:, ::3] = -0.0
    z = torch.from_numpy(z).to("cuda", TYPES[dtype][0])
    u = list(g.random(rows))
    for kw in ({}, {"k": 3}, {"k": 600}, {"k": 16000}, {"p": 0.5}, {"p": 0.123, "k": 25000}, {"m": 0.9}, {"p": 0.25, "T": 1e4}, {"k": 32999},
               {"p": 0.999999}):
        check_some(z, vocab, u=u, **kw)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_close_and_far_logits(dtype):
    """Rows whose logits are one value but for their last bits, and rows of every size."""
    rows, vocab = 258, 40000
    g = np.random.default_rng(6)
    z = 9.0 + g.integers(0, 50, (rows, vocab)) * 2.0 ** -20
    z[1::3] = g.standard_normal((rows // 3, vocab)) * 1e4
    z[2::3] = g.standard_normal((rows // 3, vocab)) * 1e-3
    z = torch.from_numpy(z).to("cuda", TYPES[dtype][0])
    u = list(g.random(rows))
    for kw in ({}, {"k": 77}, {"p": 0.37}, {"k": 3000, "p": 0.5}, {"T": 500.0, "p": 0.9}, {"k": 20000, "T": math.inf}):
        check_some(z, vocab, u=u, **kw)


@pytest.mark.parametrize("rows,fewer", [(256, (1, 2, 255)), (600, (257, 300))])
def test_bits_go_by_the_launch_shape(rows, fewer):
    """Up to 256 rows, and past 256, a row's token and the bits of its probability are the same whatever the rows beside it."""
    vocab = 20011
    z = logits_of(12, rows, vocab, "f16")
    u = list(np.random.default_rng(4).random(rows))
    for kw in ({}, {"p": 0.8}, {"k": 40}, {"k": 3000, "m": 0.001}):
        token, lp = run(z, vocab, u=u, **kw)
        for n in fewer:
            t, l = run(z[-n:], vocab, u=u[-n:], **kw)
            assert np.array_equal(t, token[-n:]) and np.array_equal(l, lp[-n:])
