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
