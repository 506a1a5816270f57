"""rq_gemm_fp8_block and its weight quantizer on the GPU against the 64-bit
oracle.

Whole numbers first: codes of -2..2 and scales of 1/2, 1 and 2 make every
product and sum exact in any order, so y has to be the rounded exact value.
Then codes of all sizes.  A y in fp32 comes from fp32 sums of exact products:
k * 2^-24 of sum |x w| bounds any order of k additions.  A 16-bit y is rounded
by half a step (2^-11, 2^-8) and, of more than 16 rows, comes from the fp8
instruction, which cuts each eight products 13 places below the largest exponent
among them: here 2^-13 of the block's largest product is allowed for each of the
128 (test_gpu_gemm_block_sums goes by the eights).
"""

import numpy as np
import pytest
import torch

import gemm_rwkv_amd.rq as rq
from oracle import codecs, next_token as nt

pytestmark = pytest.mark.gpu

OUTS = {"f16": (torch.float16, rq.RQ_F16, 2.0 ** -11), "bf16": (torch.bfloat16, rq.RQ_BF16, 2.0 ** -8),
        "f32": (torch.float32, rq.RQ_F32, 2.0 ** -24)}
B128 = rq.RQ_FP8_E4M3_B128


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def weight(wq, sw):
    n, k = wq.shape
    return rq.QWeight(B128, 0, n, k, dev(wq), dev(sw))


def run(xq, sx, wq, sw, out, ldy=None):
    dt, code, _ = OUTS[out]
    (m, k), n = xq.shape, wq.shape[0]
    ldy = ldy or n
    y = torch.full((m * ldy + 32,), 77.0, dtype=dt, device="cuda")
    x_, s_, w_ = dev(xq), dev(sx), weight(wq, sw)
    torch.cuda.synchronize()
    rq.rq_gemm_fp8_block(x_, s_, m, w_, code, y, ldy)
    torch.cuda.synchronize()
    y = y.double().cpu().numpy()
    assert (y[m * ldy:] == 77.0).all()
    y = y[:m * ldy].reshape(m, ldy)
    assert (y[:, n:] == 77.0).all()
    return y[:, :n]


def to_out(y, out):
    return torch.from_numpy(y).to(OUTS[out][0]).double().numpy()


SMALL = codecs.e4m3_encode(np.array([-2.0, -1.0, 0.0, 1.0, 2.0]))


def whole(seed, m, n, k):
    g = np.random.default_rng(seed)

    def scales(r):
        s = g.integers(126, 129, (r, nt.scale_row(k))).astype(np.uint8)
        s[:, k // 128:] = 0
        return s
    return SMALL[g.integers(0, 5, (m, k))], scales(m), SMALL[g.integers(0, 5, (n, k))], scales(-(-n // 128))


SHAPES = [(1, 1, 128), (1, 16, 128), (1, 129, 384), (1, 2048, 2048), (2, 15, 256), (3, 1000, 640), (15, 17, 1152), (16, 128, 768),
          (17, 130, 512), (31, 257, 1280), (33, 64, 2048), (48, 520, 384), (64, 1000, 256), (65, 128, 768), (100, 300, 1024),
          (127, 129, 128), (128, 256, 4096), (129, 1100, 384), (200, 2050, 768), (255, 255, 512), (257, 513, 896),
          (300, 64, 2560), (513, 384, 640), (1000, 1500, 256), (32, 8200, 1024), (5, 4096, 8192),
          # either side of each tile's border, and more than one round of tiles
          (16, 32768, 128), (16, 32752, 256), (17, 2560, 384), (40, 5130, 256), (33, 10300, 384), (70, 8100, 256), (64, 20000, 128),
          (130, 8200, 384), (260, 11000, 256), (257, 16400, 640), (1030, 11000, 384), (3100, 4100, 128), (2, 200, 65664), (70, 130, 65536),
          (1, 33, 131072), (129, 1, 1024)]


@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_whole_numbers(m, n, k, out):
    xq, sx, wq, sw = whole(m * 7 + n, m, n, k)
    want, _ = nt.product(xq, sx, wq, sw)
    assert np.array_equal(run(xq, sx, wq, sw, out), to_out(want, out))


@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("m,n,k", [(1, 300, 2048), (9, 100, 1152), (32, 1000, 768), (50, 129, 640), (128, 200, 2560), (300, 600, 1024),
                                   (40, 2048, 8192)])
def test_any_codes(m, n, k, out):
    g = np.random.default_rng(m + n)
    x = g.standard_normal((m, k)) * (1 + 30 * (g.random(k) < 0.01))
    x[m // 2, :128] = 0
    xq, sx = nt.quantize_rows(x, nt.FP8_BLOCK)
    wq, sw = nt.quantize_weight(g.standard_normal((n, k)) * k ** -0.5 * np.exp(g.standard_normal((n, 1))))
    want, size = nt.product(xq, sx, wq, sw)
    got = run(xq, sx, wq, sw, out, ldy=n + 3)
    if out == "f32":
        bound = k * 2.0 ** -24 * size
    else:
        nb = k // 128
        xm = np.abs(nt.values(xq, sx, 1)).reshape(m, nb, 128).max(-1)
        wm = np.abs(nt.values(wq, sw, 128)).reshape(n, nb, 128).max(-1)
        bound = 128 * 2.0 ** -13 * (xm @ wm.T) + k * 2.0 ** -24 * size + OUTS[out][2] * np.abs(want) * 1.01 + 2.0 ** -25
    assert (np.abs(got - want) <= bound).all(), float((np.abs(got - want) - bound).max())
    # the bounds are of the worst case; the norm of the error is what the type's rounding makes it
    assert np.linalg.norm(got - want) <= max(1.5 * OUTS[out][2], 1e-6) * np.linalg.norm(want)


def test_scales_reach_far_and_nan():
    """Scales up to 2^60 apart cancel between x and w; 0xff spoils what it scales and nothing else."""
    m, n, k = 40, 300, 512
    xq, sx, wq, sw = whole(3, m, n, k)
    shift = np.array([60, -60, 30, -60])
    sx[:, :4] = (sx[:, :4] + shift).astype(np.uint8)
    sw[:, :4] = (sw[:, :4] - shift).astype(np.uint8)
    want, _ = nt.product(xq, sx, wq, sw)
    for rows in (m, 7, 1):
        for out in OUTS:
            assert np.array_equal(run(xq[:rows], sx[:rows], wq, sw, out), to_out(want[:rows], out))
    sx[5, 2] = 255
    sw[1, 0] = 255
    for rows in (m, 7):
        for out in OUTS:
            got = run(xq[:rows], sx[:rows], wq, sw, out)
            bad = np.isnan(got)
            expect = np.zeros((rows, n), dtype=bool)
            expect[5], expect[:, 128:256] = True, True
            assert np.array_equal(bad, expect)
            assert np.array_equal(got[~bad], to_out(want[:rows], out)[~bad])


def test_rows_do_not_depend_on_each_other():
    """A row gives the same bits beside others that are not finite."""
    m, n, k = 150, 400, 640
    xq, sx, wq, sw = whole(5, m, n, k)
    clean = run(xq, sx, wq, sw, "bf16")
    xq[::2] = 0x7f
    got = run(xq, sx, wq, sw, "bf16")
    assert np.isnan(got[::2]).all() and np.array_equal(got[1::2], clean[1::2])


@pytest.mark.parametrize("n,k", [(128, 128), (200, 640), (1, 256), (300, 2048)])
def test_weight_quantizer(n, k):
    g = np.random.default_rng(n + k)
    w = (g.standard_normal((n, k)) * np.exp(3 * g.standard_normal((n, 1)))).astype(np.float32)
    w[:, :128] *= 1e-30
    if n >= 128:
        w[:128, 128 * (k // 128 - 1):] = 0
    q = rq.quantize(dev(w), B128)
    wq, sw = nt.quantize_weight(w)
    assert np.array_equal(q.codes.cpu().numpy()[:n * k].reshape(n, k), wq)
    assert np.array_equal(q.scales.cpu().numpy().reshape(sw.shape), sw)
    w[n // 2, k // 2] = np.inf
    with pytest.raises(rq.RqError) as e:
        rq.quantize(dev(w), B128)
    assert e.value.status == rq.RQ_ERR_NONFINITE


@pytest.mark.parametrize("m,n,k", [(1, 2048, 2048), (200, 512, 2048), (300, 1500, 512)])
def test_streams_and_graphs(m, n, k):
    """Two calls at once on streams of their own, and a captured one replayed on new inputs."""
    sets = [whole(s, m, n, k) for s in (1, 2)]
    wants = [to_out(nt.product(*s)[0], "f16") for s in sets]
    bufs = [[dev(s[0]), dev(s[1]), weight(s[2], s[3]), torch.zeros(m, n, dtype=torch.float16, device="cuda")] for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        for b, st in zip(bufs, streams):
            rq.rq_gemm_fp8_block(b[0], b[1], m, b[2], rq.RQ_F16, b[3], n, stream=st)
    torch.cuda.synchronize()
    for b, want in zip(bufs, wants):
        assert np.array_equal(b[3].double().cpu().numpy(), want)
    b, other = bufs
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rq.rq_gemm_fp8_block(b[0], b[1], m, b[2], rq.RQ_F16, b[3], n)
    for i in range(4):
        src = sets[i % 2]
        b[0].copy_(dev(src[0]))
        b[1].copy_(dev(src[1]))
        b[3].zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = to_out(nt.product(src[0], src[1], sets[0][2], sets[0][3])[0], "f16")
        assert np.array_equal(b[3].double().cpu().numpy(), want)


def test_far_offsets():
    """A weight of 2^31 bytes and more: the last rows come from beyond 32-bit offsets."""
    n, k = 270000, 8192
    free, _ = torch.cuda.mem_get_info()
    if free < 8 << 30:
        pytest.skip("needs 8 GiB of GPU memory")
    codes = torch.zeros(n * k, dtype=torch.uint8, device="cuda")
    scales = torch.full((-(-n // 128) * nt.scale_row(k),), 127, dtype=torch.uint8, device="cuda")
    xq, sx, wq, sw = whole(9, 3, 64, k)
    sw = np.full_like(sw, 127)
    codes[(n - 64) * k:] = dev(wq.ravel())
    w = rq.QWeight(B128, 0, n, k, codes, scales)
    y = torch.full((3, n), 5.0, dtype=torch.float16, device="cuda")
    rq.rq_gemm_fp8_block(dev(xq), dev(sx), 3, w, rq.RQ_F16, y, n)
    torch.cuda.synchronize()
    assert not y[:, :n - 64].any()
    assert np.array_equal(y[:, n - 64:].double().cpu().numpy(), to_out(nt.product(xq, sx, wq, sw)[0], "f16"))


def test_weight_quantizer_past_2_16_blocks_of_rows():
    n, k = 128 * 65600 + 5, 128
    free, _ = torch.cuda.mem_get_info()
    if free < 12 << 30:
        pytest.skip("needs 12 GiB of GPU memory")
    w = torch.zeros(n, k, device="cuda")
    g = np.random.default_rng(4)
    ends = g.standard_normal((133, k)).astype(np.float32)
    w[:128], w[-133:] = dev(ends[:128]), dev(ends)
    q = rq.quantize(w, B128)
    wq, sw = nt.quantize_weight(ends)
    codes, scales = q.codes[:n * k].view(n, k), q.scales[:-(-n // 128) * 4].view(-1, 4)
    assert np.array_equal(codes[-133:].cpu().numpy(), wq) and np.array_equal(codes[:128].cpu().numpy(), wq[:128])
    assert np.array_equal(scales[-2:].cpu().numpy(), sw) and np.array_equal(scales[0].cpu().numpy(), sw[0])
    assert not codes[128:-133].any() and not scales[1:-2].any()
