"""Draws from finite logits that lie further apart than fp32 can say, against the
64-bit oracle: tokens equal, log-probabilities as in test_gpu_sample."""

import numpy as np
import pytest
import torch

from test_gpu_sample import TYPES, check

pytestmark = pytest.mark.gpu


def rows_of(values, share, rows, vocab, dtype, seed, run=1):
    """Each logit one of `values`, taken with `share`, in runs of `run`."""
    g = np.random.default_rng(seed)
    at = g.choice(len(values), (rows, -(-vocab // run)), p=share).repeat(run, 1)[:, :vocab]
    z = np.array(values)[at]
    out = torch.full((rows, -(-vocab // 8) * 8), float("nan"), dtype=torch.float64)
    out[:, :vocab] = torch.from_numpy(z)
    return out.to("cuda", TYPES[dtype][0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [4000, 65536])
@pytest.mark.parametrize("rows", [6, 260])
def test_spread_past_fp32(rows, vocab, dtype):
    """More than a list's 512 of each value, and top_k between them, at them and past them."""
    if rows > 100 and vocab > 5000:
        vocab = 9001
    u = list(np.random.default_rng(rows).random(rows))
    low = float(torch.finfo(TYPES[dtype][0]).min)
    for values in ((1e38, -3e38), (2e38, -2e38), (3.3e38, low), (3e38, 0.0, -3e38), (3e38, 2.9e38, -2.9e38, low), (-1.0, low)):
        z = rows_of(values, [1 / len(values)] * len(values), rows, vocab, dtype, len(values), run=3)
        for k in (300, 513, 3 * vocab // 5, vocab - 1):
            check(z, vocab, k=k, u=u)
        check(z, vocab, k=3 * vocab // 5, p=0.7, T=3e38, u=u)
        check(z, vocab, k=3 * vocab // 5, T=float("inf"), u=u)
        check(z, vocab, p=0.8, T=1e38, u=u)
        check(z, vocab, p=0.999, m=0.1, T=3e38, u=u)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_few_logits_past_fp32(dtype):
    """Fewer than 512 on one side of the gap."""
    rows, vocab = 5, 3000
    u = list(np.random.default_rng(1).random(rows))
    for share in ((0.9, 0.1), (0.1, 0.9)):
        z = rows_of((1e38, -3e38), share, rows, vocab, dtype, 4)
        for k in (280, 700, 2600, 2950):
            check(z, vocab, k=k, u=u)
            check(z, vocab, k=k, T=1e38, p=0.9, u=u)


def test_classes_over_a_wide_row():
    """Logits of every size up to the largest, spread over all classes of the histogram."""
    rows, vocab = 4, 30000
    g = np.random.default_rng(7)
    for scale in (3.4e38, 1.6e38, 1e30, 1.0):
        z = torch.from_numpy((2 * g.random((rows, vocab)) - 1) * scale).float().cuda()
        u = list(g.random(rows))
        for k in (257, 5000, 20000, 29999):
            check(z, vocab, k=k, u=u)
            check(z, vocab, k=k, T=scale / 4, u=u)
            check(z, vocab, k=k, T=scale / 4, p=0.6, u=u)
