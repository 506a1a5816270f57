"""rq_sample on the GPU against the 64-bit oracle: the tokens are equal, the
log-probabilities within 1e-6 + 2^-23 of theirs (fp64 sums, one rounding to
fp32; the weights are exact to 2^-46)."""

import math

import numpy as np
import pytest
import torch

import gemm_rwkv_amd.rq as rq
from oracle import next_token as nt

pytestmark = pytest.mark.gpu

TYPES = {"f16": (torch.float16, rq.RQ_F16), "bf16": (torch.bfloat16, rq.RQ_BF16), "f32": (torch.float32, rq.RQ_F32)}


def run(logits, vocab, T=None, k=None, p=None, m=None, u=None, stream=None):
    """(tokens, logprobs) of a [rows][ld] tensor; parameters: one number or a list."""
    rows, ld = logits.shape
    code = {t[0]: t[1] for t in TYPES.values()}[logits.dtype]

    def par(v, dt=torch.float32):
        if v is None:
            return None
        v = [v] * rows if np.isscalar(v) else list(v)
        return torch.tensor(v, dtype=dt, device="cuda")
    args = par(T), par(k, torch.int32), par(p), par(m), par(u)
    token = torch.full((rows + 4,), 1234, dtype=torch.int32, device="cuda")
    logprob = torch.full((rows + 4,), 5.0, device="cuda")
    torch.cuda.synchronize()
    rq.rq_sample(code, logits, rows, vocab, ld, *args, token, logprob, stream=stream)
    torch.cuda.synchronize()
    assert (token[rows:] == 1234).all() and (logprob[rows:] == 5.0).all()
    return token[:rows].cpu().numpy(), logprob[:rows].cpu().numpy()


def f32(v):
    return float(np.float32(v))


def check(logits, vocab, T=None, k=None, p=None, m=None, u=0.0):
    rows = logits.shape[0]
    got, lp = run(logits, vocab, T, k, p, m, u)
    z = logits[:, :vocab].double().cpu().numpy()

    def at(v, i, default):
        return default if v is None else f32(v if np.isscalar(v) else v[i])
    for i in range(rows):
        want, wlp = nt.sample(z[i], at(T, i, 1.0), at(k, i, 0), at(p, i, 1.0), at(m, i, 0.0), at(u, i, 0.0))
        assert got[i] == want, (i, got[i], want, lp[i], wlp)
        if math.isinf(wlp):
            assert lp[i] == wlp
        else:
            assert abs(lp[i] - wlp) <= 1e-6 + 2.0 ** -23 * abs(wlp), (i, lp[i], wlp)


def logits_of(seed, rows, vocab, dtype, scale=2.0, ld=None):
    g = np.random.default_rng(seed)
    z = g.standard_normal((rows, ld or -(-vocab // 8) * 8)) * scale - 3
    z[np.arange(rows)[:, None], g.integers(0, vocab, (rows, 6))] += 8 * g.random((rows, 6))
    return torch.from_numpy(z).to("cuda", TYPES[dtype][0])


FILTERS = {"plain": {}, "k": {"k": 40}, "p": {"p": 0.8}, "m": {"m": 0.05}, "kp": {"k": 100, "p": 0.9}, "kpm": {"k": 30, "p": 0.95, "m": 0.02},
           "wide p": {"p": 0.9999}, "wide k": {"k": 5000}, "hot": {"T": 30.0, "p": 0.7}, "cold": {"T": 0.02}, "greedy": {"T": 0.0, "k": 5}}


@pytest.mark.parametrize("filters", FILTERS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", [(3, 7), (5, 1000), (4, 4097), (6, 50277), (3, 65536), (2, 131072)])
def test_draws(rows, vocab, dtype, filters):
    g = np.random.default_rng(vocab + len(filters))
    kw = dict(FILTERS[filters])
    check(logits_of(vocab, rows, vocab, dtype), vocab, u=list(g.random(rows)), **kw)


@pytest.mark.parametrize("dtype", TYPES)
def test_a_batch_with_parameters_of_its_own_each(dtype):
    rows, vocab = 96, 20011
    g = np.random.default_rng(8)
    check(logits_of(2, rows, vocab, dtype), vocab, T=list(np.where(g.random(rows) < 0.1, 0, 0.3 + 1.5 * g.random(rows))),
          k=[int(v) for v in np.where(g.random(rows) < 0.5, np.exp(g.random(rows) * 9).astype(int), 0)],
          p=list(np.where(g.random(rows) < 0.5, g.random(rows), 1.0)), m=list(np.where(g.random(rows) < 0.5, 0.2 * g.random(rows), 0)),
          u=list(g.random(rows)))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("levels", [1, 2, 5, 40])
def test_ties(dtype, levels):
    """Rows of a few values: borders fall between equal logits."""
    rows, vocab = 12, 9000
    g = np.random.default_rng(levels)
    z = g.integers(0, levels, (rows, 9000)).astype(np.float64) * 0.25
    z[:, ::3] = -0.0
    z = torch.from_numpy(z).to("cuda", TYPES[dtype][0])
    u = list(g.random(rows))
    for kw in ({}, {"k": 3}, {"k": 4500}, {"p": 0.5}, {"p": 0.123, "k": 7000}, {"m": 0.9}, {"T": 0.0}, {"p": 0.25, "T": 1e4},
               {"k": 8999}, {"k": 9000}, {"p": 0.999999}):
        check(z, vocab, u=u, **kw)


@pytest.mark.parametrize("vocab", [1, 2, 8, 9, 63, 64, 513])
def test_small_vocabularies(vocab):
    rows = 40
    z = logits_of(vocab, rows, vocab, "f32")
    u = [i / rows for i in range(rows)]
    for kw in ({}, {"k": 1}, {"k": 2, "p": 0.6}, {"p": 0.0}, {"p": 1.0 - 2.0 ** -24}, {"m": 1.0}, {"m": 5.0}, {"T": 0.1}):
        check(z, vocab, u=u, **kw)


@pytest.mark.parametrize("dtype", TYPES)
def test_masks_and_what_is_not_finite(dtype):
    vocab = 1500
    z = logits_of(4, 10, vocab, dtype)
    inf = float("inf")
    low = torch.finfo(TYPES[dtype][0]).min
    z[0, :] = -inf                      # nothing
    z[1, :] = float("nan")              # nothing
    z[2, :] = -inf
    z[2, 700] = 1.0                     # one
    z[3, 5:] = low                      # masked by the type's lowest value
    z[4, :] = low                       # a row of nothing else
    z[5, 3], z[5, 900] = inf, inf
    z[6, ::2] = float("nan")
    z[7, 10:] = -inf
    z[8, 1] = inf
    z[8, 2] = float("nan")
    u = list(np.random.default_rng(1).random(10))
    for kw in ({}, {"k": 5}, {"p": 0.7}, {"k": 1400, "p": 0.9}, {"m": 0.3}, {"T": 0.0}, {"T": inf}, {"T": 1e-40}, {"T": 1e30, "p": 0.5},
               {"T": inf, "p": 0.5, "k": 20}):
        check(z, vocab, u=u, **kw)


def test_numbers_outside_their_range():
    vocab = 300
    z = logits_of(5, 8, vocab, "f32")
    nan, inf = float("nan"), float("inf")
    check(z, vocab, u=[nan, -1.0, 1.0, 2.0, inf, -inf, 0.0, 1 - 2.0 ** -24])
    check(z, vocab, T=[nan, -1.0, -inf, 0.0, 1e-45, 3e38, inf, 1.0], u=[0.4] * 8)
    check(z, vocab, p=[nan, -1.0, 0.0, 1.0, 7.0, inf, -inf, 1e-30], u=[0.6] * 8)
    check(z, vocab, m=[nan, -1.0, 0.0, 1.0, 7.0, inf, -inf, 1e-30], u=[0.6] * 8)
    check(z, vocab, k=[-2 ** 31, -1, 0, 1, 299, 300, 301, 2 ** 31 - 1], u=[0.6] * 8)


def test_close_logits():
    """Values that differ in their last bits, and a row around zero with denormals."""
    g = np.random.default_rng(6)
    vocab = 6000
    a = 9.0 + g.integers(0, 50, vocab) * 2.0 ** -20
    b = g.standard_normal(vocab) * 1e-40
    c = g.standard_normal(vocab) * 1e4
    z = torch.from_numpy(np.stack([a, b, c])).float().cuda()
    u = [0.3, 0.7, 0.9]
    for kw in ({}, {"k": 77}, {"p": 0.37}, {"k": 3000, "p": 0.5}, {"T": 500.0, "p": 0.9}):
        check(z, vocab, u=u, **kw)


def test_largest_vocabulary():
    vocab = 1 << 20
    z = logits_of(3, 2, vocab, "f16")
    for kw in ({}, {"k": 50}, {"p": 0.9}):
        check(z, vocab, u=[0.2, 0.99], **kw)


def test_strided_rows_read_no_further():
    """Columns past the vocabulary hold what would win."""
    rows, vocab, ld = 6, 1003, 1200
    z = logits_of(7, rows, vocab, "bf16", ld=ld)
    z[:, vocab:] = float("inf")
    check(z, vocab, p=0.9, u=list(np.random.default_rng(2).random(rows)))


def test_many_rows_are_as_one():
    rows, vocab = 700, 2000
    z = logits_of(11, rows, vocab, "f16")
    u = list(np.random.default_rng(3).random(rows))
    got, lp = run(z, vocab, p=0.9, k=100, u=u)
    for i in (0, 255, 256, 699):
        one, l1 = run(z[i:i + 1], vocab, p=0.9, k=100, u=u[i:i + 1])
        assert one[0] == got[i] and l1[0] == lp[i]


def test_no_logprob_stream_and_graph():
    rows, vocab = 9, 65536
    z = logits_of(12, rows, vocab, "f16")
    u, T = torch.rand(rows, device="cuda"), torch.full((rows,), 0.8, device="cuda")
    p, k = torch.full((rows,), 0.9, device="cuda"), torch.full((rows,), 64, dtype=torch.int32, device="cuda")
    token = torch.empty(rows, dtype=torch.int32, device="cuda")

    def go(stream=None):
        rq.rq_sample(rq.RQ_F16, z, rows, vocab, vocab, T, k, p, None, u, token, None, stream=stream)

    go()
    torch.cuda.synchronize()
    want = token.clone()
    side = torch.cuda.Stream()
    token.zero_()
    torch.cuda.synchronize()
    go(side)
    torch.cuda.synchronize()
    assert torch.equal(token, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    for seed in range(4):
        z.copy_(logits_of(seed, rows, vocab, "f16"))
        u.copy_(torch.rand(rows, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        got = token.clone()
        go()
        torch.cuda.synchronize()
        assert torch.equal(token, got)


@pytest.mark.parametrize("dtype", TYPES)
def test_min_p_where_many_floats_weigh_the_same(dtype):
    """A min_p at or near 1 beside a largest logit of 0, or a temperature under
    which any two logits weigh the same, where some 2^30 floats lie between the
    largest and the first that weighs less; more rows than one launch shape."""
    for rows, vocab in ((4, 1000), (300, 70)):
        z = logits_of(3, rows, vocab, dtype, scale=1.0)
        z[0::4] = 0.0
        z[1::4] -= z[1::4].amax(1, keepdim=True)
        T = [1.0, 0.7, 1e30, math.inf] * (rows // 4)
        u = list(np.random.default_rng(4).random(rows))
        for m in (1.0, 2.0, 1.0 - 2.0 ** -24, 0.999, 1e-30):
            check(z, vocab, T=T, m=m, u=u)
            check(z, vocab, T=T, k=vocab - 1, p=0.9999, m=m, u=u)
