"""The time-mix operators where their arithmetic is at its edges, against the
64-bit oracle; tolerances as derived in test_gpu_mix.py."""

import numpy as np
import pytest
import torch

import gemm_rwkv_amd.rq as rq
from gemm_rwkv_amd import time_mix as tm
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


# two and four rows per workgroup, with one and two vectors of a row per thread
@pytest.mark.parametrize("code", TYPES, ids=IDS)
@pytest.mark.parametrize("lens", [[700, 0, 600], [1300], [900, 0, 801]], ids=str)
@pytest.mark.parametrize("width,nmix", [(2568, 3), (4104, 2), (8192, 1)])
def test_many_wide_rows(lens, width, nmix, code):
    t, n, ld = sum(lens), len(lens), width + 8
    say("many wide rows", lens, width, nmix, code)
    g = np.random.default_rng(t + width + 2)
    x, delta = (rows(3 * g.standard_normal((t, width)) + 1, code, ld) for _ in range(2))
    shift, dsh = (rows(g.standard_normal((n, width)), code, width) for _ in range(2))
    pd = [torch.from_numpy(z.astype(np.float32)).cuda() for z in (g.standard_normal(width), g.standard_normal(width),
                                                                  g.random((nmix, width)))]
    par = [z.double().cpu().numpy() for z in pd]
    xo, out = Out(t, width, ld, code), Out(nmix * t, width, ld, code)
    new = torch.full((n, width), float("nan"), dtype=shift[0].dtype, device="cuda")
    rq.rq_shift_norm(code, x[0], delta[0], -0.75, t, width, ld, offsets(lens), n, pd[0], pd[1], 1e-5, pd[2], nmix, shift[0],
                     new, None, n, xo.ptr(), out.ptr(), ld)
    torch.cuda.synchronize()
    wx, wo, last = mix.shift_norm(x[1], delta[1], -0.75, lens, par[0], par[1], 1e-5, par[2], shift[1])
    close(xo.get(), wx, code, "x")
    close(out.get(), wo.reshape(nmix * t, width), code, "out")
    close(new, last, code, "shift")
    # in place: the row left behind replaces the one that the first row read
    out2, same = Out(nmix * t, width, ld, code), shift[0].clone()
    rq.rq_shift_norm(code, x[0], delta[0], -0.75, t, width, ld, offsets(lens), n, pd[0], pd[1], 1e-5, pd[2], nmix, same, same,
                     None, n, None, out2.ptr(), ld)
    torch.cuda.synchronize()
    assert torch.equal(out2.get(), out.get()) and torch.equal(same, new)
    # the gradient
    up, dout = rows(g.standard_normal((t, width)), code, ld), rows(g.standard_normal((nmix * t, width)), code, ld)
    dx, din = Out(t, width, ld, code), Out(n, width, width, code)
    f32 = dict(dtype=torch.float32, device="cuda")
    dg, db, dm = (torch.full(s, float("nan"), **f32) for s in ((width,), (width,), (nmix, width)))
    rq.rq_shift_norm_backward(code, x[0], 0.5, t, width, ld, offsets(lens), n, pd[0], pd[1], 1e-5, pd[2], nmix, shift[0],
                              dout[0], ld, up[0], dsh[0], dx.ptr(), None, din.ptr(), dg, db, dm)
    torch.cuda.synchronize()
    want = mix.shift_norm_backward(x[1], lens, par[0], par[1], 1e-5, par[2], shift[1], dout[1].reshape(nmix, t, width), up[1], dsh[1])
    close(dx.get(), want["dx"], code, "dx")
    close(din.get(), want["dshift_in"], code, "dshift_in")
    for z, q in ((dg, "dgamma"), (db, "dbeta"), (dm, "dmu")):
        close(z, want[q], code, q)


# one value of one row: at a chunk's ends and inside, at the last token, in a
# partial chunk, in a short sequence, and in a first, a middle and the last
# segment of a long one
@pytest.mark.parametrize("code", TYPES, ids=IDS)
@pytest.mark.parametrize("what", ["r", "w", "k", "v", "a", "b"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")], ids=["nan", "inf"])
@pytest.mark.parametrize("lens,heads,at", [([40], 2, (16, 19, 31, 36, 39)), ([32, 20], 2, (31, 32)), ([10], 2, (4,)),
                                           ([1030], 1, (5, 700, 1029))], ids=["one", "two", "short", "long"])
def test_values_that_are_not_finite(lens, heads, at, bad, what, code):
    """They reach the outputs that the recurrence leads them to, and none of the
    tokens before."""
    t, c, n = sum(lens), 64 * heads, len(lens)
    dev, val, g = mix_inputs(lens, heads, code, c, 73)
    state = g.standard_normal((n, heads, 64, 64)).astype(np.float32)
    sd, cu = torch.from_numpy(state).cuda(), offsets(lens)
    for i in at:
        say("not finite", lens, what, bad, i, code)
        d, v = dict(dev, **{what: dev[what].clone()}), dict(val, **{what: val[what].copy()})
        d[what][i, 5], v[what][i, 5] = bad, bad
        y, out = Out(t, c, c, code), torch.empty_like(sd)
        rq.rq_time_mix(code, *(d[q] for q in "rwkvab"), t, heads, c, cu, n, sd, out, None, n, y.ptr(), c)
        torch.cuda.synchronize()
        with np.errstate(all="ignore"):
            wy, ws = mix.time_mix(*(v[q] for q in "rwkvab"), lens, state)
        for got, want, name in ((y.get(), wy, "y"), (out, ws, "state")):
            fine = np.isfinite(want)
            assert np.array_equal(torch.isfinite(got).cpu().numpy(), fine), (name, i)
            if fine.any():
                close(got.cpu()[torch.from_numpy(fine)], want[fine], code, name)


@pytest.mark.parametrize("code", TYPES, ids=IDS)
def test_rows_that_are_nowhere_finite(code):
    """From the first token on that is not finite to the end."""
    heads, lens = 2, [300]
    dev, val, g = mix_inputs(lens, heads, code, 128, 74)
    say("nowhere finite", code)
    for z in dev.values():
        z[37:] = float("nan")
    y = Out(300, 128, 128, code)
    rq.rq_time_mix(code, *(dev[q] for q in "rwkvab"), 300, heads, 128, None, 1, None, None, None, 0, y.ptr(), 128)
    torch.cuda.synchronize()
    wy, _ = mix.time_mix(*(val[q][:37] for q in "rwkvab"), [37])
    close(y.get()[:37], wy, code, "y")
    assert bool(torch.isnan(y.get()[37:]).all())


def test_gradients_of_other_heads_stay():
    """A value that is not finite takes no other head's gradients with it."""
    code, heads, lens = rq.RQ_BF16, 3, [50]
    dev, _, g = mix_inputs(lens, heads, code, 192, 75)
    dy, cu = rows(g.standard_normal((50, 192)), code, 192)[0], offsets(lens)
    say("gradients of other heads")
    got = []
    for bad in (False, True):
        d = {q: z.clone() for q, z in dev.items()}
        if bad:
            for z in d.values():
                z[20:, 64:128] = float("nan")
        outs = [torch.empty(50, 192, dtype=torch.bfloat16, device="cuda") for _ in range(6)]
        din = torch.empty(1, heads, 64, 64, device="cuda")
        rq.rq_time_mix_backward(code, *(d[q] for q in "rwkvab"), 50, heads, 192, cu, 1, None, dy, None, *outs, din)
        got.append([z[:, q] for z in outs for q in (slice(0, 64), slice(128, 192))] + [din[:, 0], din[:, 2]])
    for a, b in zip(*got):
        assert torch.isfinite(a).all() and torch.equal(a, b)


def test_torch_functions_on_two_streams():
    """Calls that cut their sequence and sum partial rows, side by side: as alone."""
    t, c = 2048, 256
    dev, _, g = mix_inputs([t], 4, rq.RQ_F16, c, 76)
    cu, f32 = offsets([t]), dict(dtype=torch.float32, device="cuda")
    param = [torch.randn(c, **f32) for _ in range(3)]
    say("torch functions on two streams")

    def go():
        leaves = [dev[q].clone().requires_grad_(True) for q in "rwkvab"]
        ps = [p.clone().requires_grad_(True) for p in param]
        y, st = tm.time_mix(*leaves, cu)
        out = tm.head_gate(y, *leaves[:1], *leaves[2:5], *ps)
        _, mixes, _ = tm.shift_norm(out, None, torch.full((6, c), 0.25, **f32), ps[0], ps[1], cu)
        (mixes.float().sum() + out.float().square().sum() + st.sum()).backward()
        return [y.detach(), st.detach(), out.detach()] + [z.grad for z in leaves + ps]

    want = go()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(go())
    torch.cuda.synchronize()
    for outs in got:
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
