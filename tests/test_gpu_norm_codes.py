"""Codes of rq_norm_quantize that are those of the 64-bit h, byte for byte.

x' = x + alpha delta has at most 35 bits (24 of alpha, 11 of a value, their lowest
places less than 2^18 apart), so fp64 holds it.  The sums and h are fp64 as well: an
h is off by some 2^-42 of itself, and a border between two codes lies within that of
one h in 2^38.  With a sum or an h in fp32 (2^-24) that is one in 2^20, and of some
millions of values several would get another code: the rows are that many.
"""

import numpy as np
import pytest
import torch

import gemm_rwkv_amd.rq as rq
from oracle import next_token as nt
from test_gpu_norm_quant import FORMATS, TYPES, call, rows

pytestmark = pytest.mark.gpu

EPS = float(np.float32(1e-5))


def quantized(h, fmt):
    """The oracle's codes and scales, many rows at a time (its scales, then its rounding by table)."""
    r, c = h.shape
    if fmt == rq.RQ_FP8_E4M3_B128:
        most = np.abs(h).reshape(r, -1, 128).max(-1)
        part, e = np.frexp(most / 448.0)
        e = np.where(most > 0, np.where(part == 0.5, e - 1, e), -127).clip(-127, 127)
        scales = np.zeros((r, nt.scale_row(c)), dtype=np.uint8)
        scales[:, :c // 128] = e + 127
        q = h * np.exp2(-e.astype(float)).repeat(128, 1)
    else:
        scales = (np.abs(h).max(1) / (127.0 if fmt == rq.RQ_I8_CH else 448.0)).astype(np.float32)
        q = h / scales.astype(float)[:, None]
        if fmt == rq.RQ_I8_CH:
            return np.clip(np.rint(q), -127, 127).astype(np.int8).view(np.uint8), scales
    # to a multiple of a code's step, ties to even; the step of [2^e, 2^(e + 1)) is 2^(e - 3), of all below 2^-6 2^-9
    step = np.exp2(np.maximum(np.frexp(q)[1] - 1, -6) - 3.0)
    v = np.minimum(np.abs(np.rint(q / step) * step), 448.0)
    e = np.maximum(np.frexp(v)[1] - 1, -6)
    code = np.where(v < 2.0 ** -6, v * 512, (e + 7) * 8 + (v / np.exp2(e.astype(float)) - 1) * 8).astype(np.uint8)
    return code | (np.signbit(q) * 128).astype(np.uint8), scales


def test_quantized_is_the_oracles():
    g = np.random.default_rng(1)
    h = g.standard_normal((5, 512)) * np.exp2(g.integers(-20, 20, (5, 1)))
    h[1] = np.round(g.standard_normal(512) * 16) / 16
    for fmt in FORMATS:
        for a, b in zip(quantized(h, fmt), nt.quantize_rows(h, fmt)):
            assert np.array_equal(a, b)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("alpha", [0.1, 0.7071067811865476, 1.0, -1.0 / 3.0])
@pytest.mark.parametrize("dtype,m,width", [("f16", 700, 4096), ("bf16", 500, 2560), ("f16", 60, 16384), ("bf16", 90, 8192)])
def test_sums_with_the_residual(dtype, m, width, alpha, fmt):
    dt, alpha = TYPES[dtype][0], float(np.float32(alpha))
    x, delta = rows(m, m, width, dt), rows(m + 1, m, width, dt, 0.7)
    codes, scales = call(x, delta, alpha, width, rq.RQ_NORM_NONE, None, None, 0.0, fmt)
    h = x.double().cpu().numpy() + alpha * delta.double().cpu().numpy()
    want, wscale = quantized(h, fmt)
    assert np.array_equal(scales, wscale)
    assert np.array_equal(codes, want), int((codes != want).sum())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", [rq.RQ_NORM_RMS, rq.RQ_NORM_LAYER], ids=["rms", "layer"])
@pytest.mark.parametrize("m,width,parts", [(1500, 4096, "g"), (3000, 4096, "gb"), (700, 4096, ""), (300, 2560, "gb"), (1, 2048, "gb"),
                                           (200, 8192, "gb"), (100, 16384, "g")])
def test_normed_rows(m, width, parts, kind, fmt):
    g = np.random.default_rng(m + width)
    half = g.integers(1, 9, (m, width // 2)) * g.choice([-1, 1], (m, width // 2))
    x = np.concatenate([half, -half], 1)
    x[:, width // 4] *= 20
    x[:, width // 4 + width // 2] *= 20
    for row in x:
        g.shuffle(row)
    x = x.astype(np.float64)
    assert (x ** 2).sum(1).max() < 2 ** 24 and not x.sum(1).any()
    gamma = (1 + 0.2 * g.standard_normal(width)).astype(np.float32) if "g" in parts else None
    beta = (0.1 * g.standard_normal(width)).astype(np.float32) if "b" in parts else None
    d = [None if v is None else torch.from_numpy(v).cuda() for v in (gamma, beta)]
    codes, scales = call(torch.from_numpy(x).half().cuda(), None, 0.0, width, kind, *d, EPS, fmt)
    h = nt.normed(x, kind, None if gamma is None else gamma.astype(float), None if beta is None else beta.astype(float), EPS)
    want, wscale = quantized(h, fmt)
    assert np.array_equal(scales, wscale)
    assert np.array_equal(codes, want), int((codes != want).sum())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", [rq.RQ_NORM_RMS, rq.RQ_NORM_LAYER], ids=["rms", "layer"])
@pytest.mark.parametrize("dtype,m,width,alpha,mean", [("f16", 1700, 4096, 0.3, 0.0), ("bf16", 1500, 2560, None, 4.0), ("f16", 700, 8192, 1.0, 300.0),
                                                      ("bf16", 200, 16384, -0.7, 0.5), ("f16", 5000, 272, 0.5, 1.0), ("bf16", 3000, 640, None, 0.0)])
def test_any_rows(dtype, m, width, alpha, mean, kind, fmt):
    if fmt == rq.RQ_FP8_E4M3_B128 and width % 128:
        width = 256
    dt, g = TYPES[dtype][0], np.random.default_rng(m)
    x = rows(m, m, width, dt) + mean
    delta = None if alpha is None else rows(m + 1, m, width, dt, 0.6)
    alpha = 0.0 if alpha is None else float(np.float32(alpha))
    gamma = (1 + 0.2 * g.standard_normal(width)).astype(np.float32)
    beta = (0.1 * g.standard_normal(width)).astype(np.float32) if kind == rq.RQ_NORM_LAYER else None
    d = [None if v is None else torch.from_numpy(v).cuda() for v in (gamma, beta)]
    codes, scales = call(x, delta, alpha, width, kind, *d, EPS, fmt)
    full = x.double().cpu().numpy()
    if delta is not None:
        full = full + alpha * delta.double().cpu().numpy()
    h = nt.normed(full, kind, gamma.astype(float), None if beta is None else beta.astype(float), EPS)
    want, wscale = quantized(h, fmt)
    assert np.array_equal(scales, wscale), int((scales != wscale).sum())
    assert np.array_equal(codes, want), int((codes != want).sum())


@pytest.mark.parametrize("width", [640, 4096, 6016])
@pytest.mark.parametrize("with_beta", [False, True])
@pytest.mark.parametrize("fmt", FORMATS)
def test_rows_of_one_value(fmt, with_beta, width):
    """Their variance is 0 and h is beta alone, exactly; without one the scales and codes are those of zeros."""
    g = np.random.default_rng(3)
    x = torch.from_numpy(np.repeat(g.standard_normal((20, 1)) * 10, width, 1)).half().cuda()
    beta = (0.1 * g.standard_normal(width)).astype(np.float32)
    codes, scales = call(x, None, 0.0, width, rq.RQ_NORM_LAYER, None, torch.from_numpy(beta).cuda() if with_beta else None, EPS, fmt)
    if with_beta:
        want, wscale = nt.quantize_rows(beta[None].astype(float).repeat(20, 0), fmt)
        assert np.array_equal(codes, want) and np.array_equal(scales, wscale)
    else:
        assert not (codes & 127).any() and not scales.any()


@pytest.mark.parametrize("fmt,most", [(rq.RQ_FP8_E4M3_CH, 448.0), (rq.RQ_I8_CH, 127.0)])
def test_scale_of_the_largest_in_all_its_bits(fmt, most):
    """Rows whose largest |h|, its bits rounded to 53 of 64 as a double of them would be, gives another scale in fp32."""
    alpha, g = float(np.float32(0.1)), np.random.default_rng(5)
    gamma = (1 + 0.2 * g.standard_normal(16)).astype(np.float32)
    v = (1024 + np.arange(1024)) / 1024.0
    found = []
    for j in range(16):
        h = (v[:, None] + alpha * v) * float(gamma[j])
        rounded = h.view(np.uint64).astype(np.float64).astype(np.uint64).view(np.float64)
        found += [(j, v[a], v[b]) for a, b in np.argwhere((h / most).astype(np.float32) != (rounded / most).astype(np.float32))]
    assert len(found) >= 4
    x, delta = np.zeros((2, len(found), 16))
    for r, (j, a, b) in enumerate(found):
        x[r, j], delta[r, j] = a, b
    h = (x + alpha * delta) * gamma.astype(float)
    _, scales = call(torch.from_numpy(x).half().cuda(), torch.from_numpy(delta).half().cuda(), alpha, 16, rq.RQ_NORM_NONE,
                     torch.from_numpy(gamma).cuda(), None, 0.0, fmt)
    assert np.array_equal(scales, (h.max(1) / most).astype(np.float32))


@pytest.mark.parametrize("fmt", FORMATS)
def test_sums_past_fp32(fmt):
    """x' beyond fp32 is infinite in x_out, and counts for h where a gamma brings it back; an h beyond fp32 is not finite."""
    width = 256
    x, delta = torch.zeros(3, width).to("cuda", torch.bfloat16), rows(4, 3, width, torch.bfloat16, 0.02)
    delta[1] = torch.linspace(-3e38, 3e38, width).to("cuda", torch.bfloat16)
    x_out = torch.empty_like(x)
    for gamma, finite in ((1e-4, True), (1.0, False)):
        gv = torch.full((width,), gamma, device="cuda")
        codes, scales = call(x, delta, 16.0, width, rq.RQ_NORM_NONE, gv, None, 0.0, fmt, x_out)
        h = 16.0 * delta.double().cpu().numpy() * float(np.float32(gamma))
        assert torch.isinf(x_out[1]).any() and not torch.isinf(x_out[[0, 2]]).any()
        if not finite:
            h[1] = np.where(np.abs(h[1]) >= 2.0 ** 128, np.inf, h[1])
        want, wscale = nt.quantize_rows(h, fmt)
        assert np.array_equal(scales, wscale, equal_nan=fmt != rq.RQ_FP8_E4M3_B128)
        assert np.array_equal(codes, want)
