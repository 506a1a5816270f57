"""The state recurrence on whole numbers: every product and sum of these inputs
is a whole number below 2^24, so that fp32 holds it exactly, in any order, and
what is stored must be the exact value rounded once.  The numbers that are
multiplied have 18 bits and cancel to a few: whoever keeps fewer than fp32's 24
bits of a state, a product of two rows or a removed value misses by whole units.

The decays are exactly 1 (a raw decay of -6e4, whose sigmoid is 0)."""

import numpy as np
import pytest
import torch

import gemm_rwkv_amd.rq as rq
from gpu_helpers import say
from oracle import mix

pytestmark = pytest.mark.gpu

TORCH = {rq.RQ_F16: torch.float16, rq.RQ_BF16: torch.bfloat16}
TYPES, IDS = [rq.RQ_F16, rq.RQ_BF16], ["f16", "bf16"]


def forward_inputs(kind, tokens, nseq, heads, g):
    """Rows (heads joined) and states.  Tokens come in pairs that take back what
    they add, up to a small d."""
    x = {q: np.zeros((tokens, heads, 64)) for q in "rkvab"}
    x["w"] = np.full((tokens, heads, 64), -6e4)
    S = np.zeros((nseq, heads, 64, 64))
    pair, odd = np.arange(tokens) // 2, np.arange(tokens) % 2
    big = lambda *s: g.integers(1 << 17, 1 << 18, s)     # 18 bits
    few = lambda *s: g.integers(0, 4, s)
    sign = (1 - 2 * odd)[:, None, None]
    rows = np.zeros((tokens, heads, 2))                  # 1000 hi + lo has 18 bits, from channels of eight
    rows[:, :, 0] = g.integers(128, 256, (tokens, heads))[2 * pair]
    rows[:, :, 1] = g.integers(4, 256, (tokens, heads))[2 * pair] - odd[:, None] * few(tokens, heads)
    if kind == "state":            # y = S r
        n = big(nseq, heads, 64, 32)
        S[..., 0::2], S[..., 1::2] = n, n - few(nseq, heads, 64, 32)
        s = 1 - 2 * g.integers(0, 2, (tokens, heads, 32))
        x["r"][..., 0::2], x["r"][..., 1::2] = s, -s
    elif kind == "keys":           # y = sum v (k r)
        x["k"][..., :2] = rows
        x["v"][:] = sign * g.integers(1, 4, (heads, 64))
        x["r"][..., 0], x["r"][..., 1] = 1000 * odd[:, None], odd[:, None]
    elif kind == "removals":       # y = sum u (b r)
        S[..., 5] = g.integers(1, 4, (nseq, heads, 64))
        x["a"][..., 5:6] = sign
        x["b"][..., :2] = rows
        x["r"][..., 0], x["r"][..., 1] = 1000 * odd[:, None], odd[:, None]
    else:                          # "removed": the same with large u
        n = big(nseq, heads, 64)
        S[..., 5], S[..., 6] = n, n - few(nseq, heads, 64)
        x["a"][..., 5], x["a"][..., 6] = 1 - odd[:, None], -odd[:, None]
        x["b"][..., 0] = 1
        x["r"][..., 0] = odd[:, None]
    return {q: z.reshape(tokens, -1) for q, z in x.items()}, S


def device_rows(x, code):
    d = torch.from_numpy(np.ascontiguousarray(x)).cuda().to(TORCH[code])
    return d, d.double().cpu().numpy()


def exactly(got, want, what):
    assert np.array_equal(want, np.rint(want)) and np.abs(want).max(initial=0) < 1 << 24
    w = torch.from_numpy(want).to(got.dtype).reshape(got.shape)
    bad = got.cpu() != w
    assert not bool(bad.any()), (what, int(bad.sum()), got.cpu()[bad][:4], w[bad][:4])


@pytest.mark.parametrize("code", TYPES, ids=IDS)
@pytest.mark.parametrize("kind", ["state", "keys", "removals", "removed"])
@pytest.mark.parametrize("lens,heads", [([2], 2), ([16], 2), ([70], 3), ([34, 2, 0, 40], 2), ([1030], 1)], ids=str)
def test_outputs(lens, heads, kind, code):
    say("exact", kind, lens, heads, code)
    t, n, c = sum(lens), len(lens), 64 * heads
    g = np.random.default_rng(t)
    rows, S = forward_inputs(kind, t, n, heads, g)
    dev, val = {}, {}
    for q, z in rows.items():
        dev[q], val[q] = device_rows(z, code)
        assert q == "w" or np.array_equal(z, val[q])
    y, out = torch.empty(t, c, dtype=TORCH[code], device="cuda"), torch.empty(n, heads, 64, 64, device="cuda")
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    rq.rq_time_mix(code, *(dev[q] for q in "rwkvab"), t, heads, c, cu, n, torch.from_numpy(S).float().cuda(), out, None, n, y, c)
    torch.cuda.synchronize()
    wy, ws = mix.time_mix(*(val[q] for q in "rwkvab"), lens, S)
    exactly(y, wy, "y")
    exactly(out, ws, "state")


def backward_inputs(kind, tokens, nseq, heads, g):
    """Rows with dy, states and their gradients; what is large comes in pairs
    that differ by a small d and are read with opposite signs."""
    x = {q: np.zeros((tokens, heads, 64)) for q in "rkvab"}
    x["w"], x["dy"] = np.full((tokens, heads, 64), -6e4), np.zeros((tokens, heads, 64))
    S, D = np.zeros((nseq, heads, 64, 64)), np.zeros((nseq, heads, 64, 64))
    pair, odd = np.arange(tokens) // 2, np.arange(tokens) % 2
    sign, even = (1 - 2 * odd)[:, None, None], (1 - odd)[:, None]
    few = lambda *s: g.integers(0, 4, s)
    rows = np.zeros((tokens, heads, 2))
    rows[:, :, 0] = g.integers(128, 256, (tokens, heads))[2 * pair]
    rows[:, :, 1] = g.integers(4, 256, (tokens, heads))[2 * pair] - odd[:, None] * few(tokens, heads)

    def pairs(axis):               # [v][k] of 18 bits, paired along an axis
        n = np.repeat(g.integers(1 << 17, 1 << 18, (nseq, heads, 64, 64)), 2, axis)
        n = n.take(np.arange(64), axis)
        low = few(nseq, heads, 64, 64) * (np.arange(64) % 2).reshape((64, 1) if axis == 2 else (1, 64))
        return n - low

    def signs(rows_):              # s, -s, s, -s ...
        s = np.repeat(1 - 2 * g.integers(0, 2, (rows_, heads, 32)), 2, -1)
        return s * (1 - 2 * (np.arange(64) % 2))

    if kind == "dr of states":
        S, x["dy"] = pairs(2), signs(tokens)
    elif kind == "dv of states":
        D, x["k"] = pairs(3), signs(tokens)
    elif kind == "dk of states":
        D, x["v"] = pairs(2), signs(tokens)
    elif kind == "db of states":
        D, S[..., 5] = pairs(2), signs(nseq)
        x["a"][..., 5] = 1
    elif kind == "da of states":
        S, D[..., 7] = pairs(2), signs(nseq)
        x["b"][..., 7] = 1
    elif kind == "dr of removed":
        S[..., 5], x["dy"] = pairs(2)[..., 5], signs(tokens)
        x["a"][..., 5] = 1
        x["b"][..., :1] = sign
    elif kind == "dk of products":
        x["v"][..., 0], x["v"][..., 1] = 1000 * even, even
        x["dy"][..., :2] = rows
        x["r"][:] = sign * g.integers(1, 4, (heads, 64))
    elif kind == "dv of products":
        x["k"][..., 0], x["k"][..., 1] = 1000 * even, even
        x["r"][..., :2] = rows
        x["dy"][:] = sign * g.integers(1, 4, (heads, 64))
    else:                          # "dk of removed"
        D[..., 7], x["v"] = pairs(2)[..., 7], signs(tokens)
        x["b"][..., 7] = 1
        x["a"][..., :1] = sign
    return {q: z.reshape(tokens, -1) for q, z in x.items()}, S, D


KINDS = ["dr of states", "dv of states", "dk of states", "db of states", "da of states", "dr of removed", "dk of products",
         "dv of products", "dk of removed"]


@pytest.mark.parametrize("code", TYPES, ids=IDS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,heads", [([2], 2), ([16], 2), ([70], 3), ([34, 2, 0, 40], 2)], ids=str)
def test_gradients(lens, heads, kind, code):
    say("exact", kind, lens, heads, code)
    t, n, c = sum(lens), len(lens), 64 * heads
    g = np.random.default_rng(t)
    rows, S, D = backward_inputs(kind, t, n, heads, g)
    dev, val = {}, {}
    for q, z in rows.items():
        dev[q], val[q] = device_rows(z, code)
        assert q == "w" or np.array_equal(z, val[q])
    outs = [torch.empty(t, c, dtype=TORCH[code], device="cuda") for _ in range(6)]
    sd, dd = (torch.from_numpy(z).float().cuda() for z in (S, D))
    din = torch.empty_like(sd)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    rq.rq_time_mix_backward(code, *(dev[q] for q in "rwkvab"), t, heads, c, cu, n, sd, dev["dy"], dd, *outs, din)
    torch.cuda.synchronize()
    want = mix.time_mix_backward(*(val[q] for q in "rwkvab"), lens, S, val["dy"], D)
    for o, q in zip(outs, ("dr", "dw", "dk", "dv", "da", "db")):
        exactly(o, want[q], q)
    exactly(din, want["dstate"], "dstate")
