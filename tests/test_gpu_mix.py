"""The time-mix operators on the GPU against the 64-bit oracle (oracle/mix.py):
sequences of lengths 0, 1 and around every tile edge, both 16-bit types,
strides, states in slots, streams, graphs and repeats.

Tolerances.  A 16-bit output is rounded once, by at most u = 2^-11 (fp16) or
2^-8 (bf16, eight significant bits) of its value; everything before is fp32.
The recurrence adds at most a dozen fp32 roundings of 2^-24 per token to a
state whose norm a token does not raise, so after T <= 1100 tokens their
random sum is within sqrt(12 * 1100) * 2^-24 = 6.8e-6 of it; 2e-5 bounds the
relative L2 error of every fp32 output and the fp32 share of every 16-bit one.
Single elements may cancel: on top of u |value| they are held to 1e-3 of the
array's root mean square, which is 2e-5 times sqrt(64) (a sum over a head's
channels) with a margin of six."""

import numpy as np
import pytest
import torch

import gemm_rwkv_amd.rq as rq
from gpu_helpers import Guarded, say
from oracle import mix

pytestmark = pytest.mark.gpu

U = {rq.RQ_F16: 2.0 ** -11, rq.RQ_BF16: 2.0 ** -8}
TINY = {rq.RQ_F16: 2.0 ** -25, rq.RQ_BF16: 2.0 ** -134}
TORCH = {rq.RQ_F16: torch.float16, rq.RQ_BF16: torch.bfloat16}
FP32_L2 = 2e-5
FP32_ELEM = 1e-3
TYPES = [rq.RQ_F16, rq.RQ_BF16]
IDS = ["f16", "bf16"]


def close(got, want, code, what):
    """got: torch tensor; want: float64 numpy of the same size."""
    g = got.detach().double().cpu().numpy().reshape(want.shape)
    assert np.isfinite(g).all(), what
    if want.size == 0:
        return
    u, tiny = (U[code], TINY[code]) if got.dtype != torch.float32 else (2.0 ** -24, 2.0 ** -149)
    rms = np.sqrt((want * want).mean())
    d = np.abs(g - want)
    l2 = np.sqrt((d * d).sum()) / max(np.sqrt((want * want).sum()), 1e-300)
    assert l2 <= u + FP32_L2 + (tiny / rms if rms else 0), (what, "l2", l2)
    worst = (d - (u * np.abs(want) + FP32_ELEM * rms + tiny)).max()
    assert worst <= 0, (what, "element", worst, rms)


def rows(x, code, ld):
    """[tokens][ld] device rows of the values x, NaN between the rows; and the
    16-bit values as float64."""
    t, c = x.shape
    d = torch.full((t, ld), float("nan"), dtype=TORCH[code], device="cuda")
    d[:, :c] = torch.from_numpy(x).cuda().to(TORCH[code])
    return d, d[:, :c].double().cpu().numpy()


class Out:
    """Output rows inside a guarded buffer, NaN before the call."""

    def __init__(self, t, c, ld, code):
        self.g, self.c = Guarded(t * ld * 2), c
        self.full = self.g.t.view(TORCH[code]).view(t, ld)
        self.full.fill_(float("nan"))

    def ptr(self):
        return self.full.data_ptr()

    def get(self):
        # nothing around or between the rows was written
        self.g.check_guards()
        assert bool(torch.isnan(self.full[:, self.c:]).all())
        return self.full[:, :self.c]


def offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def mix_inputs(lens, heads, code, ld, seed, raw=None):
    g = np.random.default_rng(seed)
    t, c = int(sum(lens)), 64 * heads
    kap = g.standard_normal((t, heads, 64)) + 0.7 * g.standard_normal((1, heads, 64))
    kap /= np.linalg.norm(kap, axis=-1, keepdims=True)
    rate = 1 / (1 + np.exp(-g.standard_normal((t, heads, 64))))
    x = {"r": g.standard_normal((t, c)), "w": g.standard_normal(c) * 2 - 1.5 + g.standard_normal((t, c)) * 0.5,
         "k": 0.5 * g.standard_normal((t, c)), "v": g.standard_normal((t, c)), "a": -kap.reshape(t, c),
         "b": (kap * rate).reshape(t, c)}
    if raw is not None:
        x["w"] = np.broadcast_to(raw, (t, c)).copy()
    dev, val = {}, {}
    for q, z in x.items():
        dev[q], val[q] = rows(z, code, ld)
    return dev, val, g


LENS = [[1], [2], [15], [16], [17], [31, 33], [0, 5, 0, 1, 40, 0], [64, 1, 65], [300], [1025], [7] * 20]


@pytest.mark.parametrize("code", TYPES, ids=IDS)
@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("ws", [None, False], ids=["ws", "none"])
def test_time_mix(lens, code, ws):
    check_time_mix(lens, 1 if max(lens) > 500 else 3, code, ws)


# several sequences cut into segments; batches of mostly short sequences, of
# which some, or none, are longer than the step kernel takes there
@pytest.mark.parametrize("code", TYPES, ids=IDS)
@pytest.mark.parametrize("lens,heads", [([700, 0, 900], 2), ([1, 24, 25, 0, 70, 2] * 8, 6), ([3] * 300, 1)],
                         ids=["segments", "short and long", "short"])
def test_time_mix_batches(lens, heads, code):
    check_time_mix(lens, heads, code, None)


def check_time_mix(lens, heads, code, ws):
    c, ld = 64 * heads, 64 * heads + 8
    t, n = sum(lens), len(lens)
    say("time_mix", lens, code, heads, ws)
    dev, val, g = mix_inputs(lens, heads, code, ld, 1 + t)
    nslots = n + 3
    slots = g.permutation(nslots)[:n].astype(np.int32)
    pool = g.standard_normal((nslots, heads, 64, 64)).astype(np.float32)
    pd = torch.from_numpy(pool).cuda()
    sd = torch.from_numpy(slots).cuda()
    y = Out(t, c, ld, code)
    args = [dev[q] for q in "rwkvab"]
    rq.rq_time_mix(code, *args, t, heads, ld, offsets(lens), n, pd, pd, sd, nslots, y.ptr(), ld, ws=ws)
    torch.cuda.synchronize()
    wy, ws_ = mix.time_mix(*(val[q] for q in "rwkvab"), lens, pool[slots].astype(np.float64))
    close(y.get(), wy, code, "y")
    close(pd[sd.long()], ws_, code, "state")
    rest = np.setdiff1d(np.arange(nslots), slots)
    assert np.array_equal(pd.cpu().numpy()[rest], pool[rest])          # the other slots are as they were
    # the same call again, out of place and without slots: the same bits
    order = torch.from_numpy(pool[slots]).cuda()
    out = torch.full_like(order, float("nan"))
    y2 = Out(t, c, ld, code)
    rq.rq_time_mix(code, *args, t, heads, ld, offsets(lens), n, order, out, None, n, y2.ptr(), ld, ws=ws)
    assert torch.equal(y2.get(), y.get()) and torch.equal(out, pd[sd.long()])
    # no states at all: zeros, and none kept
    y3 = Out(t, c, ld, code)
    rq.rq_time_mix(code, *args, t, heads, ld, offsets(lens), n, None, None, None, 0, y3.ptr(), ld, ws=ws)
    wy, _ = mix.time_mix(*(val[q] for q in "rwkvab"), lens)
    close(y3.get(), wy, code, "y from zeros")


@pytest.mark.parametrize("code", TYPES, ids=IDS)
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_time_mix_backward(lens, code):
    heads = 1 if max(lens) > 500 else 3
    c, ld = 64 * heads, 64 * heads + 16
    t, n = sum(lens), len(lens)
    say("time_mix_backward", lens, code, heads)
    dev, val, g = mix_inputs(lens, heads, code, ld, 101 + t)
    dyd, dy = rows(g.standard_normal((t, c)), code, ld)
    state = g.standard_normal((n, heads, 64, 64)).astype(np.float32)
    ds = (0.1 * g.standard_normal((n, heads, 64, 64))).astype(np.float32)
    for full in (True, False):
        outs = [Out(t, c, ld, code) for _ in range(6)]
        din = torch.full((n, heads, 64, 64), float("nan"), device="cuda")
        sd, dsd = (torch.from_numpy(x).cuda() if full else None for x in (state, ds))
        rq.rq_time_mix_backward(code, *(dev[q] for q in "rwkvab"), t, heads, ld, offsets(lens), n, sd, dyd, dsd,
                                *(o.ptr() for o in outs), din if full else None)
        torch.cuda.synchronize()
        want = mix.time_mix_backward(*(val[q] for q in "rwkvab"), lens, state if full else np.zeros_like(state), dy,
                                     ds if full else None)
        for o, q in zip(outs, ("dr", "dw", "dk", "dv", "da", "db")):
            close(o.get(), want[q], code, q)
        if full:
            close(din, want["dstate"], code, "dstate")


@pytest.mark.parametrize("raw", [-60000.0, -3.0, 60000.0], ids=["keeps", "slow", "fastest"])
@pytest.mark.parametrize("lens", [[70], [33, 2]], ids=str)
def test_time_mix_extreme_decays(raw, lens):
    """Decays of exactly 1 and of the least value, exp(-exp(-1/2)), throughout."""
    code, heads = rq.RQ_F16, 2
    t, c, n = sum(lens), 128, len(lens)
    say("time_mix decays", raw, lens)
    dev, val, g = mix_inputs(lens, heads, code, c, 7, raw)
    dyd, dy = rows(g.standard_normal((t, c)), code, c)
    state = g.standard_normal((n, heads, 64, 64)).astype(np.float32)
    sd, so = torch.from_numpy(state).cuda(), torch.empty(n, heads, 64, 64, device="cuda")
    y = Out(t, c, c, code)
    rq.rq_time_mix(code, *(dev[q] for q in "rwkvab"), t, heads, c, offsets(lens), n, sd, so, None, n, y.ptr(), c)
    wy, wst = mix.time_mix(*(val[q] for q in "rwkvab"), lens, state)
    close(y.get(), wy, code, "y")
    close(so, wst, code, "state")
    outs = [Out(t, c, c, code) for _ in range(6)]
    rq.rq_time_mix_backward(code, *(dev[q] for q in "rwkvab"), t, heads, c, offsets(lens), n, sd, dyd, None,
                            *(o.ptr() for o in outs), so)
    want = mix.time_mix_backward(*(val[q] for q in "rwkvab"), lens, state, dy)
    for o, q in zip(outs, ("dr", "dw", "dk", "dv", "da", "db")):
        close(o.get(), want[q], code, q)
    close(so, want["dstate"], code, "dstate")


def test_time_mix_scales():
    """bf16 rows far from one: keys of 1e-12, values of 1e12, receptances of
    1e9, and a repeated removal direction (its products do not cancel)."""
    code, heads, lens = rq.RQ_BF16, 1, [50]
    say("time_mix scales")
    dev, val, g = mix_inputs(lens, heads, code, 64, 9)
    scale = {"r": 1e9, "w": 1, "k": 1e-12, "v": 1e12, "a": 1, "b": 1}
    one = g.standard_normal((1, 64))
    one /= np.linalg.norm(one)
    for q in scale:
        x = np.repeat(-one if q == "a" else one, 50, 0) if q in "ab" else val[q] * scale[q]
        dev[q], val[q] = rows(x, code, 64)
    so = torch.empty(1, 1, 64, 64, device="cuda")
    y = Out(50, 64, 64, code)
    rq.rq_time_mix(code, *(dev[q] for q in "rwkvab"), 50, 1, 64, offsets(lens), 1, None, so, None, 1, y.ptr(), 64)
    wy, wst = mix.time_mix(*(val[q] for q in "rwkvab"), lens)
    close(y.get(), wy, code, "y")
    close(so, wst, code, "state")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_sequences_do_not_leak(bad):
    """What is not finite in one sequence stays in it."""
    code, heads, lens = rq.RQ_F16, 2, [21, 30, 18]
    t, c = sum(lens), 128
    say("time_mix leak", bad)
    dev, val, g = mix_inputs(lens, heads, code, c, 11)
    x = torch.from_numpy(g.standard_normal((t, c))).cuda().half()
    hurt = {q: z.clone() for q, z in dev.items()}
    for z in hurt.values():
        z[21:51] = bad
    xh = x.clone()
    xh[21:51] = bad
    keep = torch.tensor(list(range(21)) + list(range(51, 69)), device="cuda")
    cu = offsets(lens)
    f32 = dict(dtype=torch.float32, device="cuda")
    par = [torch.randn(c, **f32), torch.randn(c, **f32), 1e-5, torch.rand(2, c, **f32)]
    got = []
    for d, z in ((dev, x), (hurt, xh)):
        y = torch.empty(t, c, dtype=torch.float16, device="cuda")
        st = torch.empty(3, heads, 64, 64, **f32)
        rq.rq_time_mix(code, *(d[q] for q in "rwkvab"), t, heads, c, cu, 3, None, st, None, 3, y, c)
        gr = [torch.empty_like(y) for _ in range(6)]
        dst = torch.empty_like(st)
        rq.rq_time_mix_backward(code, *(d[q] for q in "rwkvab"), t, heads, c, cu, 3, None, z, None, *gr, dst)
        out, sh = torch.empty(2, t, c, dtype=torch.float16, device="cuda"), torch.empty(3, c, dtype=torch.float16, device="cuda")
        rq.rq_shift_norm(code, z, None, 1.0, t, c, c, cu, 3, *par, 2, None, sh, None, 3, None, out, c)
        got.append([y[keep], st[[0, 2]], *(q[keep] for q in gr), dst[[0, 2]], out[:, keep], sh[[0, 2]]])
    for p, q in zip(*got):
        assert torch.isfinite(p).all() and torch.equal(p, q)


def test_slots_outside_the_array():
    """A sequence without a slot starts from zeros and leaves nothing; the
    others are as if it were not there."""
    code, heads, lens = rq.RQ_F16, 1, [1, 1, 20, 1]
    t, n = sum(lens), 4
    say("slots outside")
    dev, val, g = mix_inputs(lens, heads, code, 64, 12)
    pool = g.standard_normal((3, 1, 64, 64)).astype(np.float32)
    slots = np.array([2, -1, 3, 0], np.int32)
    start = np.stack([pool[2], 0 * pool[0], 0 * pool[0], pool[0]])
    wy, wst = mix.time_mix(*(val[q] for q in "rwkvab"), lens, start)
    pd, y = torch.from_numpy(pool).cuda(), Out(t, 64, 64, code)
    rq.rq_time_mix(code, *(dev[q] for q in "rwkvab"), t, 1, 64, offsets(lens), n, pd, pd, torch.from_numpy(slots).cuda(), 3,
                   y.ptr(), 64)
    close(y.get(), wy, code, "y")
    close(pd[[2, 0]], wst[[0, 3]], code, "state")
    assert np.array_equal(pd[1].cpu().numpy(), pool[1])
    f32 = dict(dtype=torch.float32, device="cuda")
    gamma, beta, mu = torch.randn(64, **f32), torch.randn(64, **f32), torch.rand(1, 64, **f32)
    shift, sv = rows(g.standard_normal((3, 64)), code, 64)
    x, xv = rows(g.standard_normal((t, 64)), code, 64)
    out = Out(t, 64, 64, code)
    new = shift.clone()
    rq.rq_shift_norm(code, x, None, 0.0, t, 64, 64, offsets(lens), n, gamma, beta, 1e-5, mu, 1, new, new,
                     torch.from_numpy(slots).cuda(), 3, None, out.ptr(), 64)
    p = [z.double().cpu().numpy() for z in (gamma, beta, mu)]
    _, wo, last = mix.shift_norm(xv, None, 0.0, lens, p[0], p[1], 1e-5, p[2], np.stack([sv[2], 0 * sv[0], 0 * sv[0], sv[0]]))
    close(out.get(), wo[0], code, "out")
    close(new[[2, 0]], last[[0, 3]], code, "shift")
    assert torch.equal(new[1], shift[1])


NORM_LENS = [[1], [5], [0, 3, 0, 1, 9, 0], [1] * 32, [37], [700, 0, 600], [900, 0, 801]]


@pytest.mark.parametrize("code", TYPES, ids=IDS)
@pytest.mark.parametrize("lens", NORM_LENS, ids=str)
@pytest.mark.parametrize("width,nmix", [(8, 1), (72, 6), (768, 6), (2568, 3), (4104, 8), (8192, 1)])
def test_shift_norm(lens, width, nmix, code):
    if sum(lens) > 1000 and width > 1000:
        pytest.skip("the oracle's share of the same paths is covered at smaller sizes")
    t, n, ld = sum(lens), len(lens), width + 8
    say("shift_norm", lens, width, nmix, code)
    g = np.random.default_rng(t + width)
    x, delta = (rows(3 * g.standard_normal((t, width)) + 1, code, ld) for _ in range(2))
    shift = rows(g.standard_normal((n, width)), code, width)
    par = [g.standard_normal(width), g.standard_normal(width), g.random((nmix, width))]
    pd = [torch.from_numpy(z.astype(np.float32)).cuda() for z in par]
    par = [z.double().cpu().numpy() for z in pd]
    xo, out = Out(t, width, ld, code), Out(nmix * t, width, ld, code)
    new = torch.full((n, width), float("nan"), dtype=TORCH[code], device="cuda")
    rq.rq_shift_norm(code, x[0], delta[0], -0.75, t, width, ld, offsets(lens), n, pd[0], pd[1], 1e-5, pd[2], nmix, shift[0],
                     new, None, n, xo.ptr(), out.ptr(), ld)
    torch.cuda.synchronize()
    wx, wo, last = mix.shift_norm(x[1], delta[1], -0.75, lens, par[0], par[1], 1e-5, par[2], shift[1])
    close(xo.get(), wx, code, "x")
    close(out.get(), wo.reshape(nmix * t, width), code, "out")
    close(new, last, code, "shift")
    # in place, no residual, nothing else kept
    out2, same = Out(nmix * t, width, ld, code), shift[0].clone()
    rq.rq_shift_norm(code, x[0], None, 1.0, t, width, ld, offsets(lens), n, pd[0], pd[1], 1e-5, pd[2], nmix, same, same,
                     None, n, None, out2.ptr(), ld)
    _, wo, last = mix.shift_norm(x[1], None, 0.0, lens, par[0], par[1], 1e-5, par[2], shift[1])
    close(out2.get(), wo.reshape(nmix * t, width), code, "out in place")
    close(same, last, code, "shift in place")


@pytest.mark.parametrize("code", TYPES, ids=IDS)
@pytest.mark.parametrize("lens", NORM_LENS, ids=str)
@pytest.mark.parametrize("width,nmix", [(8, 1), (72, 6), (768, 6), (2568, 3), (4104, 8), (8192, 1)])
@pytest.mark.parametrize("ws", [None, False], ids=["ws", "none"])
def test_shift_norm_backward(lens, width, nmix, code, ws):
    if sum(lens) > 1000 and width > 1000:
        pytest.skip("the oracle's share of the same paths is covered at smaller sizes")
    t, n, ld = sum(lens), len(lens), width + 8
    say("shift_norm_backward", lens, width, nmix, code, ws)
    g = np.random.default_rng(t + width + 1)
    x, up = rows(3 * g.standard_normal((t, width)) + 1, code, ld), rows(g.standard_normal((t, width)), code, ld)
    dout = rows(g.standard_normal((nmix * t, width)), code, ld)
    shift, dsh = (rows(g.standard_normal((n, width)), code, width) for _ in range(2))
    pd = [torch.from_numpy(z.astype(np.float32)).cuda() for z in (g.standard_normal(width), g.standard_normal(width),
                                                                  g.random((nmix, width)))]
    par = [z.double().cpu().numpy() for z in pd]
    dx, dd, din = Out(t, width, ld, code), Out(t, width, ld, code), Out(n, width, width, code)
    f32 = dict(dtype=torch.float32, device="cuda")
    dg, db, dm = (torch.full(s, float("nan"), **f32) for s in ((width,), (width,), (nmix, width)))
    rq.rq_shift_norm_backward(code, x[0], 0.5, t, width, ld, offsets(lens), n, pd[0], pd[1], 1e-5, pd[2], nmix, shift[0],
                              dout[0], ld, up[0], dsh[0], dx.ptr(), dd.ptr(), din.ptr(), dg, db, dm, ws=ws)
    torch.cuda.synchronize()
    want = mix.shift_norm_backward(x[1], lens, par[0], par[1], 1e-5, par[2], shift[1], dout[1].reshape(nmix, t, width), up[1], dsh[1])
    close(dx.get(), want["dx"], code, "dx")
    close(dd.get(), 0.5 * want["dx"], code, "ddelta")
    close(din.get(), want["dshift_in"], code, "dshift_in")
    for z, q in ((dg, "dgamma"), (db, "dbeta"), (dm, "dmu")):
        close(z, want[q], code, q)
    # without what is optional
    dx2, dg2, db2, dm2 = Out(t, width, ld, code), *(torch.empty_like(z) for z in (dg, db, dm))
    rq.rq_shift_norm_backward(code, x[0], 0.5, t, width, ld, offsets(lens), n, pd[0], pd[1], 1e-5, pd[2], nmix, None, dout[0],
                              ld, None, None, dx2.ptr(), None, None, dg2, db2, dm2, ws=ws)
    want = mix.shift_norm_backward(x[1], lens, par[0], par[1], 1e-5, par[2], None, dout[1].reshape(nmix, t, width))
    close(dx2.get(), want["dx"], code, "dx alone")
    for z, q in ((dg2, "dgamma"), (db2, "dbeta"), (dm2, "dmu")):
        close(z, want[q], code, q + " alone")


@pytest.mark.parametrize("code", TYPES, ids=IDS)
@pytest.mark.parametrize("tokens", [1, 3, 16, 17, 130, 1000])
@pytest.mark.parametrize("heads", [1, 3, 12, 40])
def test_head_gate(tokens, heads, code):
    c, ld = 64 * heads, 64 * heads + 24
    say("head_gate", tokens, heads, code)
    g = np.random.default_rng(tokens + heads)
    x = {q: rows(g.standard_normal((tokens, c)) * (2 if q == "y" else 1) + (q == "y"), code, ld) for q in "yrkvgd"}
    pd = [torch.from_numpy(g.standard_normal(c).astype(np.float32)).cuda() for _ in range(3)]
    par = [z.double().cpu().numpy() for z in pd]
    out = Out(tokens, c, ld, code)
    rq.rq_head_gate(code, *(x[q][0] for q in "yrkvg"), tokens, heads, ld, pd[0], pd[1], 64e-5, pd[2], out.ptr(), ld)
    torch.cuda.synchronize()
    close(out.get(), mix.head_gate(*(x[q][1] for q in "yrkvg"), par[0], par[1], 64e-5, par[2]), code, "out")
    want = mix.head_gate_backward(*(x[q][1] for q in "yrkvg"), par[0], par[1], 64e-5, par[2], x["d"][1])
    for ws in (None, False):
        outs = [Out(tokens, c, ld, code) for _ in range(5)]
        ps = [torch.full((c,), float("nan"), device="cuda") for _ in range(3)]
        rq.rq_head_gate_backward(code, *(x[q][0] for q in "yrkvg"), tokens, heads, ld, pd[0], pd[1], 64e-5, pd[2], x["d"][0],
                                 *(o.ptr() for o in outs), *ps, ws=ws)
        torch.cuda.synchronize()
        for o, q in zip(outs, ("dy", "dr", "dk", "dv", "dg")):
            close(o.get(), want[q], code, q)
        for z, q in zip(ps, ("dgamma", "dbeta", "du")):
            close(z, want[q], code, q)


def test_head_of_equal_values():
    """A head without variance: eps alone keeps the norm finite."""
    say("head_gate constant")
    code, c = rq.RQ_F16, 64
    y = rows(np.full((2, c), 3.0), code, c)
    one = rows(np.ones((2, c)), code, c)
    pd = [torch.ones(c, device="cuda") for _ in range(3)]
    out = Out(2, c, c, code)
    rq.rq_head_gate(code, y[0], one[0], one[0], one[0], one[0], 2, 1, c, pd[0], pd[1], 64e-5, pd[2], out.ptr(), c)
    o = np.ones(c)
    close(out.get(), mix.head_gate(y[1], *(one[1],) * 4, o, o, 64e-5, o), code, "out")


@pytest.mark.parametrize("rows_held", [8, 0], ids=["arrays", "null"])
def test_no_tokens(rows_held):
    """Empty calls carry states over and clear the parameters' gradients, also
    with the null addresses of empty tensors."""
    code, c = rq.RQ_BF16, 64
    say("no tokens", rows_held)
    f32 = dict(dtype=torch.float32, device="cuda")
    e = torch.empty(rows_held, c, dtype=torch.bfloat16, device="cuda")
    more = [torch.empty_like(e) for _ in range(6)]
    st, so = torch.randn(2, 1, 64, 64, **f32), torch.empty(2, 1, 64, 64, **f32)
    rq.rq_time_mix(code, *(e,) * 6, 0, 1, c, None, 2, st, so, None, 2, more[0], c)
    assert torch.equal(st, so)
    so.zero_()
    rq.rq_time_mix_backward(code, *(e,) * 6, 0, 1, c, None, 2, None, e, st, *more, so)
    assert torch.equal(st, so)
    sh, sn = torch.randn(2, c, device="cuda").bfloat16(), torch.empty(2, c, dtype=torch.bfloat16, device="cuda")
    w = [torch.ones(c, **f32), torch.ones(c, **f32), 1e-5, torch.ones(1, c, **f32), 1]
    rq.rq_shift_norm(code, e, None, 1.0, 0, c, c, None, 2, *w, sh, sn, None, 2, None, more[0], c)
    assert torch.equal(sh, sn)
    sn.zero_()
    gr = [torch.full((c,), 5.0, **f32) for _ in range(3)]
    rq.rq_shift_norm_backward(code, e, 1.0, 0, c, c, None, 2, *w, None, more[1], c, None, sh, more[0], None, sn, *gr)
    assert torch.equal(sh, sn) and not any(z.any() for z in gr)
    gr = [torch.full((c,), 5.0, **f32) for _ in range(3)]
    rq.rq_head_gate_backward(code, *(e,) * 5, 0, 1, c, w[0], w[1], 1e-5, w[0], e, *more[:5], *gr)
    assert not any(z.any() for z in gr)


def _everything(lens, heads, code, d, st, ws, big):
    """Every entry once, on the current stream; what they wrote."""
    t, c, n = sum(lens), 64 * heads, len(lens)
    h = dict(dtype=TORCH[code], device="cuda")
    f32 = dict(dtype=torch.float32, device="cuda")
    o = {"y": torch.empty(t, c, **h), "st": torch.empty_like(st), "x": torch.empty(t, c, **h), "mix": torch.empty(3, t, c, **h),
         "sh": torch.empty(n, c, **h), "gate": torch.empty(t, c, **h), "ds": torch.empty_like(st)}
    for i in range(13):
        o["g%d" % i] = torch.empty(t, c, **h)
    for i in range(6):
        o["p%d" % i] = torch.empty(3 if i == 2 else 1, c, **f32)

    def go():
        a = [d[q] for q in "rwkvab"]
        rq.rq_shift_norm(code, d["r"], d["k"], 0.5, t, c, c, d["cu"], n, d["p"], d["q"], 1e-5, d["mu"], 3, None, o["sh"], None, n,
                         o["x"], o["mix"], c)
        rq.rq_time_mix(code, *a, t, heads, c, d["cu"], n, st, o["st"], None, n, o["y"], c, ws=ws)
        rq.rq_head_gate(code, o["y"], d["r"], d["k"], d["v"], d["a"], t, heads, c, d["p"], d["q"], 64e-5, d["u"], o["gate"], c)
        rq.rq_head_gate_backward(code, o["y"], d["r"], d["k"], d["v"], d["a"], t, heads, c, d["p"], d["q"], 64e-5, d["u"], d["b"],
                                 *(o["g%d" % i] for i in range(5)), o["p3"], o["p4"], o["p5"], ws=ws)
        rq.rq_time_mix_backward(code, *a, t, heads, c, d["cu"], n, st, d["r"], None, *(o["g%d" % i] for i in range(5, 11)),
                                o["ds"], ws=big)
        rq.rq_shift_norm_backward(code, o["x"], 0.5, t, c, c, d["cu"], n, d["p"], d["q"], 1e-5, d["mu"], 3, None, o["mix"], c, None,
                                  None, o["g11"], o["g12"], None, o["p0"], o["p1"], o["p2"], ws=ws)
    return o, go


def test_streams_repeats_and_graph():
    """The same bits on another stream, again, and from a captured graph
    replayed between eager calls."""
    code, heads, lens = rq.RQ_F16, 4, [33, 0, 190, 1]
    t, c, n = sum(lens), 256, 4
    dev, _, g = mix_inputs(lens, heads, code, c, 21)
    f32 = dict(dtype=torch.float32, device="cuda")
    dev.update(cu=offsets(lens), p=torch.randn(c, **f32), q=torch.randn(c, **f32), mu=torch.rand(3, c, **f32), u=torch.randn(c, **f32))
    st = torch.randn(n, heads, 64, 64, **f32)
    wss = [(torch.zeros(1 << 20, dtype=torch.uint8, device="cuda"),
            torch.empty(rq.rq_time_mix_backward_bytes(t, heads, n), dtype=torch.uint8, device="cuda")) for _ in range(2)]
    say("every entry: eager")
    want, go = _everything(lens, heads, code, dev, st, *wss[0])
    go()
    torch.cuda.synchronize()
    first = {q: x.clone() for q, x in want.items()}
    for q, x in first.items():
        assert torch.isfinite(x).all(), q
    assert not wss[0][0][:65536].any()                    # the split counters are as they were
    side = torch.cuda.Stream()
    other, go_other = _everything(lens, heads, code, dev, st, *wss[1])
    torch.cuda.synchronize()
    say("every entry: another stream, beside the first")
    with torch.cuda.stream(side):
        go_other()
    go()
    torch.cuda.synchronize()
    for q in first:
        assert torch.equal(first[q], want[q]) and torch.equal(first[q], other[q]), q
    say("every entry: capture and replays")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        go_other()
    for rep in range(3):
        for x in other.values():
            x.zero_()
        go()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for q in first:
            assert torch.equal(first[q], other[q]), (rep, q)


def test_rows_past_32_bits():
    """Rows whose element offsets pass 2^32: interleaved in one array of 8.6 GB."""
    code, heads, t = rq.RQ_F16, 1, 2060
    ld = 1 << 21
    say("rows past 2^32")
    dev, val, g = mix_inputs([t], heads, code, 64, 31)
    big = torch.empty(t * ld, dtype=torch.float16, device="cuda").view(t, ld)
    src = {}
    for i, q in enumerate("rwkvab"):
        big[:, 64 * i:64 * i + 64] = dev[q]
        src[q] = big.data_ptr() + 128 * i
    y, y1, gate, gate1 = (torch.empty(t, 64, dtype=torch.float16, device="cuda") for _ in range(4))
    st, st1 = (torch.empty(1, 1, 64, 64, device="cuda") for _ in range(2))
    rq.rq_time_mix(code, *(src[q] for q in "rwkvab"), t, 1, ld, None, 1, None, st, None, 1, y, 64)
    rq.rq_time_mix(code, *(dev[q] for q in "rwkvab"), t, 1, 64, None, 1, None, st1, None, 1, y1, 64)
    assert torch.equal(y, y1) and torch.equal(st, st1)
    one = torch.ones(64, device="cuda")
    rq.rq_head_gate(code, *(src[q] for q in "rkvab"), t, 1, ld, one, one, 64e-5, one, gate, 64)
    rq.rq_head_gate(code, *(dev[q] for q in "rkvab"), t, 1, 64, one, one, 64e-5, one, gate1, 64)
    assert torch.equal(gate, gate1)
    mu = torch.rand(1, 64, device="cuda")
    rq.rq_shift_norm(code, src["r"], src["k"], 0.5, t, 64, ld, None, 1, one, one, 1e-5, mu, 1, None, None, None, 1, None, gate, 64)
    rq.rq_shift_norm(code, dev["r"], dev["k"], 0.5, t, 64, 64, None, 1, one, one, 1e-5, mu, 1, None, None, None, 1, None, gate1, 64)
    assert torch.equal(gate, gate1)


def test_offsets_that_break_the_rule():
    """Offsets outside the array or falling are clamped by the kernels' own
    bounds: nothing past the arrays is written and the calls end."""
    code, heads, t = rq.RQ_F16, 1, 40
    dev, _, g = mix_inputs([t], heads, code, 64, 41)
    one = torch.ones(64, device="cuda")
    for cu in ([0, 100, 7], [-5, 12, 90], [0, 0, 0], [30, 10, 40]):
        say("clamped offsets", cu)
        cd = torch.tensor(cu, dtype=torch.int32, device="cuda")
        gy = Guarded(t * 128)
        st = Guarded(2 * 64 * 64 * 4)
        rq.rq_time_mix(code, *(dev[q] for q in "rwkvab"), t, 1, 64, cd, 2, None, st.ptr(), None, 2, gy.ptr(), 64)
        gs = [Guarded(t * 128) for _ in range(7)]
        rq.rq_time_mix_backward(code, *(dev[q] for q in "rwkvab"), t, 1, 64, cd, 2, None, dev["r"], None,
                                *(z.ptr() for z in gs[:6]), st.ptr())
        rq.rq_shift_norm(code, dev["r"], None, 1.0, t, 64, 64, cd, 2, one, one, 1e-5, one, 1, None, None, None, 2, None,
                         gs[6].ptr(), 64)
        p = [Guarded(256) for _ in range(3)]
        rq.rq_shift_norm_backward(code, dev["r"], 1.0, t, 64, 64, cd, 2, one, one, 1e-5, one, 1, None, dev["k"], 64, None, None,
                                  gs[6].ptr(), None, None, *(z.ptr() for z in p))
        torch.cuda.synchronize()
        for z in [gy, st] + gs + p:
            z.check_guards()
