"""rq_norm_quantize on the GPU against the 64-bit oracle.

Where h is the input itself (no norm, no residual, no parameters) codes and
scales are the oracle's byte for byte.  Elsewhere the bound here is what an h in
fp32 would need: its sums have at most 64 sequential terms per thread and 8 per
workgroup, its roots and quotients one rounding each, so with S = |n gamma| + |gamma|
mean|x| / rms + |beta| such an h is off by less than 128 * 2^-24 S = 2^-17 S.  (The
kernel's is fp64; test_gpu_norm_codes holds it to that.)  A code's value is off by
half a step more: 2^-4 of h in e4m3 (2^-10 of the scale where it is subnormal), half
the scale in int8.
"""

import numpy as np
import pytest
import torch

import gemm_rwkv_amd.rq as rq
from oracle import codecs, next_token as nt

pytestmark = pytest.mark.gpu

TYPES = {"f16": (torch.float16, rq.RQ_F16, 2.0 ** -11), "bf16": (torch.bfloat16, rq.RQ_BF16, 2.0 ** -8)}
FORMATS = (rq.RQ_FP8_E4M3_CH, rq.RQ_I8_CH, rq.RQ_FP8_E4M3_B128)
GUARD = 0xA5


def rows(seed, m, n, dt, scale=1.0, ld=None):
    g = np.random.default_rng(seed)
    x = g.standard_normal((m, ld or n)) * scale
    x[:, n // 3] *= 30.0
    return torch.from_numpy(x).to("cuda", dt)


def scale_bytes(m, width, fmt):
    return m * nt.scale_row(width) if fmt == rq.RQ_FP8_E4M3_B128 else 4 * m


def call(x, delta, alpha, width, kind, gamma, beta, eps, fmt, x_out=None, stream=None):
    """(codes [rows][width], scales) with guards behind both checked."""
    m, ld = x.shape
    code = {t[0]: t[1] for t in TYPES.values()}[x.dtype]
    nb = scale_bytes(m, width, fmt)
    codes = torch.full((m * width + 64,), GUARD, dtype=torch.uint8, device="cuda")
    scales = torch.full((nb + 64,), GUARD, dtype=torch.uint8, device="cuda")
    if stream is not None:
        torch.cuda.synchronize()
    rq.rq_norm_quantize(code, kind, x, delta, alpha, m, width, ld, gamma, beta, eps, fmt, x_out, codes, scales, stream=stream)
    torch.cuda.synchronize()
    codes, scales = codes.cpu().numpy(), scales.cpu().numpy()
    assert (codes[m * width:] == GUARD).all() and (scales[nb:] == GUARD).all()
    codes, scales = codes[:m * width].reshape(m, width), scales[:nb].copy()
    return codes, scales.reshape(m, -1) if fmt == rq.RQ_FP8_E4M3_B128 else scales.view(np.float32)


def check(codes, scales, h, slop, fmt):
    """Codes and scales against h, known to within slop."""
    width = h.shape[1]
    if fmt == rq.RQ_FP8_E4M3_B128:
        nb = width // 128
        assert not scales[:, nb:].any()
        step = np.exp2(scales[:, :nb].astype(float) - 127).repeat(128, 1)
        most = np.abs(h).reshape(-1, nb, 128).max(-1)
        off = slop.reshape(-1, nb, 128).max(-1)
        e = scales[:, :nb].astype(float) - 127
        assert (448 * np.exp2(e) >= most - off).all()
        assert ((448 * np.exp2(e - 1) < most + off) | (e == -127)).all()
    else:
        most = np.abs(h).max(1)
        want = most / (127 if fmt == rq.RQ_I8_CH else 448)
        assert (np.abs(scales - want) <= 2.0 ** -23 * want + slop.max(1) / 127).all()
        step = scales.astype(float)[:, None]
    vals = codes.view(np.int8).astype(float) if fmt == rq.RQ_I8_CH else codecs.e4m3_decode(codes)
    # the scale's own rounding makes the largest quotient 448 (1 + 2^-24)
    half = 0.5 * step if fmt == rq.RQ_I8_CH else np.maximum(2.0 ** -4 * np.abs(h), 2.0 ** -10 * step)
    err = np.abs(vals * step - h)
    assert (err <= half * (1 + 2.0 ** -16) + slop + 1e-40).all(), float((err - half - slop).max())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,width", [(1, 128), (3, 768), (5, 4096), (2, 4224), (2, 8192), (1, 8320), (1, 16384)])
def test_codes_are_exact_without_a_norm(m, width, dtype, fmt):
    dt = TYPES[dtype][0]
    x = rows(width + m, m, width, dt)
    x[0, :128] *= 1e-4
    if m > 2:
        x[1] = 0
        x[2, 128:256] = 0
    h = x.double().cpu().numpy()
    codes, scales = call(x, None, 0.0, width, rq.RQ_NORM_NONE, None, None, 0.0, fmt)
    want, wscale = nt.quantize_rows(h, fmt)
    assert np.array_equal(scales, wscale)
    assert np.array_equal(codes, want)


@pytest.mark.parametrize("fmt", FORMATS[:2])
def test_same_bytes_as_quantize_act(fmt):
    """Halves whose quotients fall on ties, nearly on ties, and anywhere."""
    g = np.random.default_rng(5)
    m, width = 64, 1024
    a = np.concatenate([g.integers(-448, 449, (m // 2, width)) / 16.0, g.standard_normal((m - m // 2, width))])
    a *= np.exp2(g.integers(-12, 3, (m, 1)))
    x = torch.from_numpy(a).to("cuda", torch.float16)
    codes, scales = call(x, None, 0.0, width, rq.RQ_NORM_NONE, None, None, 0.0, fmt)
    want = torch.empty(m * width, dtype=torch.uint8, device="cuda")
    ws = torch.empty(m, dtype=torch.float32, device="cuda")
    rq.rq_quantize_act(x, m, width, width, fmt, want, ws)
    assert np.array_equal(scales, ws.cpu().numpy())
    assert np.array_equal(codes.ravel(), want.cpu().numpy())


@pytest.mark.parametrize("most", [1e-38, 3e-43, 1e30])
def test_scales_at_the_ends_of_fp32(most):
    x = (rows(3, 4, 256, torch.float32) / 100 * most).to(torch.bfloat16)
    h = x.double().cpu().numpy()
    for fmt in FORMATS:
        codes, scales = call(x, None, 0.0, 256, rq.RQ_NORM_NONE, None, None, 0.0, fmt)
        want, wscale = nt.quantize_rows(h, fmt)
        assert np.array_equal(scales, wscale), fmt
        assert np.array_equal(codes, want), fmt


@pytest.mark.parametrize("kind", [rq.RQ_NORM_NONE, rq.RQ_NORM_RMS, rq.RQ_NORM_LAYER])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m,width,dtype,parts", [(1, 2048, "f16", "dgbx"), (7, 128, "bf16", "dx"), (33, 2560, "bf16", "gb"),
                                                 (2, 16384, "f16", "dgx"), (3, 8192, "f16", "gbd"), (5, 640, "f16", "")])
def test_norms(m, width, dtype, parts, fmt, kind):
    dt, _, half = TYPES[dtype]
    ld = width + 24
    x = rows(width * 3 + m, m, width, dt, 1.5, ld)
    delta = rows(width + 1, m, width, dt, 1.0, ld) if "d" in parts else None
    g = np.random.default_rng(m)
    gamma = torch.from_numpy(1 + 0.2 * g.standard_normal(width)).float().cuda() if "g" in parts else None
    beta = torch.from_numpy(0.1 * g.standard_normal(width)).float().cuda() if "b" in parts else None
    x_out = torch.full((m, ld), 7.0, dtype=dt, device="cuda") if "x" in parts else None
    codes, scales = call(x, delta, 0.5, width, kind, gamma, beta, 1e-5, fmt, x_out)
    full = x[:, :width].double().cpu().numpy()
    if delta is not None:
        full = full + 0.5 * delta[:, :width].double().cpu().numpy()
    gn = None if gamma is None else gamma.double().cpu().numpy()
    bn = None if beta is None else beta.double().cpu().numpy()
    h = nt.normed(full, kind, gn, bn, 1e-5)
    ag = np.ones(width) if gn is None else np.abs(gn)
    ab = np.zeros(width) if bn is None else np.abs(bn)
    spread = np.abs(nt.normed(full, kind, None, None, 1e-5))
    rel = np.abs(full).mean(1, keepdims=True) / np.sqrt((full * full).mean(1, keepdims=True)) if kind == rq.RQ_NORM_LAYER else 0.0
    check(codes, scales, h, 2.0 ** -17 * (spread * ag + ag * rel + ab), fmt)
    if x_out is not None:
        got = x_out.double().cpu().numpy()
        assert (got[:, width:] == 7.0).all()
        assert (np.abs(got[:, :width] - full) <= np.abs(full) * (half + 2.0 ** -23) + 1e-7).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_many_rows_in_place(fmt):
    """Runs of several rows per workgroup; x_out replaces x; codes equal those
    of the same rows on their own."""
    m, width = 9001, 256
    x, delta = rows(1, m, width, torch.float16), rows(2, m, width, torch.float16)
    gamma = torch.rand(width, device="cuda") + 0.5
    keep = x.clone()
    codes, scales = call(x, delta, 1.0, width, rq.RQ_NORM_LAYER, gamma, None, 1e-5, fmt, x)
    assert torch.equal(x, (keep.float() + delta.float()).half())
    for at in (0, 1, 4096, 8999, 9000):
        c1, s1 = call(keep[at:at + 1].clone(), delta[at:at + 1].clone(), 1.0, width, rq.RQ_NORM_LAYER, gamma, None, 1e-5, fmt)
        assert np.array_equal(c1[0], codes[at]) and np.array_equal(s1[0], scales[at])


@pytest.mark.parametrize("kind", [rq.RQ_NORM_NONE, rq.RQ_NORM_RMS, rq.RQ_NORM_LAYER])
def test_what_is_not_finite(kind):
    m, width = 6, 512
    x = rows(9, m, width, torch.bfloat16)
    x[1, 200] = float("nan")
    x[2, 300] = float("inf")
    x[3, 10] = -float("inf")
    x[4] = 3e38        # finite, but its squares are not
    for fmt in FORMATS:
        codes, scales = call(x, None, 0.0, width, kind, None, None, 1e-5, fmt)
        clean, cscales = call(x[[0, 5]].contiguous(), None, 0.0, width, kind, None, None, 1e-5, fmt)
        assert np.array_equal(codes[[0, 5]], clean) and np.array_equal(scales[[0, 5]], cscales)
        if fmt == rq.RQ_FP8_E4M3_B128:
            bad = scales[:, :4] == 255
            want = {1: 1, 2: 2, 3: 0}
            for i, b in want.items():
                assert bad[i, b]
                if kind == rq.RQ_NORM_NONE:
                    assert bad[i].sum() == 1
            assert bad[4].all() == (kind != rq.RQ_NORM_NONE)
            assert not codes[bad.repeat(128, 1)].any()
        else:
            bad = np.isnan(scales)
            assert bad.tolist() == [False, True, True, True, kind != rq.RQ_NORM_NONE, False]
            assert not codes[bad].any()


def test_stream_and_graph():
    m, width = 5, 2048
    x, gamma = rows(4, m, width, torch.float16), torch.rand(width, device="cuda")
    codes = torch.zeros(m, width, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(m, 16, dtype=torch.uint8, device="cuda")
    x_out, delta = torch.empty_like(x), rows(5, m, width, torch.float16)

    def go(stream=None):
        rq.rq_norm_quantize(rq.RQ_F16, rq.RQ_NORM_RMS, x, delta, 1.0, m, width, width, gamma, None, 1e-5,
                            rq.RQ_FP8_E4M3_B128, x_out, codes, scales, stream=stream)

    go()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = codes.clone(), scales.clone()
    codes.zero_()
    torch.cuda.synchronize()
    go(side)
    torch.cuda.synchronize()
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    for seed in range(3):
        x.copy_(rows(seed, m, width, torch.float16))
        g.replay()
        torch.cuda.synchronize()
        got = codes.clone(), scales.clone()
        go()
        torch.cuda.synchronize()
        assert torch.equal(codes, got[0]) and torch.equal(scales, got[1])
