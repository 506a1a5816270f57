"""Rows with +inf, which alone can be drawn, all equal: top_k keeps the first of
them by index however they lie over the row's parts.  Against the 64-bit oracle."""

import numpy as np
import pytest
import torch

from test_gpu_sample import TYPES, check, logits_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", [(8, 1500), (8, 65536), (264, 9001)])
def test_first_of_many_infinities(rows, vocab, dtype):
    """No other logit is -inf, so the row's smallest is finite; the infinities lie in
    one part of the row, in a few, everywhere, or are fewer than top_k."""
    inf = float("inf")
    z = logits_of(vocab, rows, vocab, dtype)
    g = np.random.default_rng(3)
    z[0::8, vocab // 2:vocab // 2 + 400] = inf
    z[1::8, ::7] = inf
    z[2::8, :vocab] = inf
    z[3::8, vocab - 3:vocab] = inf
    z[4::8, torch.from_numpy(g.permutation(vocab)[:300]).cuda()] = inf
    z[5::8, :64] = inf
    z[5::8, vocab - 64:vocab] = inf
    z[6::8, 700] = inf
    z[7::8, ::2] = inf
    z[7::8, 1::2] = -inf               # and one kind of row with both
    u = list(g.random(rows))
    for k in (1, 2, 40, 256, 257, 1000):
        check(z, vocab, k=k, u=u)
    check(z, vocab, k=100, p=0.5, m=0.5, u=u)
    check(z, vocab, u=u)
    check(z, vocab, p=0.3, u=u)
