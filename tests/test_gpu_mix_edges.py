"""The time-mix operators where their arithmetic is at its edges, against the
64-bit oracle; tolerances as derived in test_gpu_mix.py."""

import numpy as np
import pytest
import torch

import gemm_rwkv_amd.rq as rq
from gpu_helpers import say
from oracle import mix
from test_gpu_mix import IDS, TYPES, Out, close, mix_inputs, offsets, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("code", TYPES, ids=IDS)
@pytest.mark.parametrize("raw", [-16.0, -10.0, 8.0, 10.0, 13.0, 16.0])
def test_gradient_of_flat_decays(raw, code):
    """Raw decays far out on the sigmoid, where its slope is small beside 1:
    the decay's gradient keeps its relative accuracy.  (dy is scaled up, so
    that the gradient stays inside fp16.)"""
    heads, lens = 2, [37, 3]
    t, c, n = sum(lens), 128, 2
    say("flat decays", raw, code)
    dev, val, g = mix_inputs(lens, heads, code, c, 71, raw)
    dyd, dy = rows(100 * g.standard_normal((t, c)), code, c)
    state = g.standard_normal((n, heads, 64, 64)).astype(np.float32)
    outs = [Out(t, c, c, code) for _ in range(6)]
    rq.rq_time_mix_backward(code, *(dev[q] for q in "rwkvab"), t, heads, c, offsets(lens), n, torch.from_numpy(state).cuda(), dyd,
                            None, *(o.ptr() for o in outs), None)
    torch.cuda.synchronize()
    want = mix.time_mix_backward(*(val[q] for q in "rwkvab"), lens, state, dy)
    for o, q in zip(outs, ("dr", "dw", "dk", "dv", "da", "db")):
        close(o.get(), want[q], code, q)


def test_gradient_on_given_streams():
    """The launch stream as an argument, as an object, a handle and the null
    stream, between calls on the current one: the same bits."""
    code, heads, lens = rq.RQ_F16, 2, [300, 41]
    t, c, n = sum(lens), 128, 2
    say("gradient on given streams")
    dev, _, g = mix_inputs(lens, heads, code, c, 72)
    dy, cu = rows(g.standard_normal((t, c)), code, c)[0], offsets(lens)

    def go(**kw):
        outs = [torch.empty(t, c, dtype=torch.float16, device="cuda") for _ in range(6)]
        torch.cuda.synchronize()
        for _ in range(3):
            rq.rq_time_mix_backward(code, *(dev[q] for q in "rwkvab"), t, heads, c, cu, n, None, dy, None, *outs, None, **kw)
        return outs

    want, side = go(), torch.cuda.Stream()
    for kw in ({"stream": side}, {}, {"stream": side.cuda_stream}, {"stream": 0}):
        got = go(**kw)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), kw
    with torch.cuda.stream(side):
        got = go(stream=0)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
