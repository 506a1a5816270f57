"""What the torch functions of the time-mixing layer refuse before the library
is called, which takes bare addresses.  Nothing runs on a GPU here: the
library's entries are stand-ins that fail the test when they are reached."""

import pytest
import torch

from gemm_rwkv_amd import time_mix as tm

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
T, C, N = 6, 128, 2
CU = tm.offsets([4, 2], "cpu")


@pytest.fixture(autouse=True)
def library(monkeypatch):
    for name in ("rq_shift_norm", "rq_time_mix", "rq_head_gate", "rq_fused_rkv", "rq_gemm_small_m", "rq_gemm_w4"):
        def reached(*args, _name=name, **kw):
            pytest.fail(_name + " was reached")
        monkeypatch.setattr(tm.rq, name, reached)


def rows(dtype=F16, t=T, c=C):
    return torch.zeros(t, c, dtype=dtype)


def f32(*shape):
    return torch.zeros(*shape)


MIX = dict({q: rows() for q in "rwkvab"}, cu=CU, state=f32(N, 2, 64, 64))
NORM = dict(x=rows(), delta=rows(), mu=f32(3, C), gamma=f32(C), beta=f32(C), cu=CU, shift=rows(t=N))
GATE = dict({q: rows() for q in "yrkvg"}, gamma=f32(C), beta=f32(C), u=f32(C))

BAD_CU = [("cu", CU.long(), TypeError), ("cu", CU[None], ValueError), ("cu", CU[:0], ValueError)]
BAD = [(tm.time_mix, MIX, *bad) for bad in
       [(q, z, e) for q in "wkvab" for z, e in ((rows(F32), TypeError), (rows(BF16), TypeError), (rows(t=T - 1), ValueError),
                                               (rows(c=64), ValueError), (rows()[0], ValueError))] +
       [("r", rows(F32), TypeError), ("r", rows()[0], ValueError)] + BAD_CU +
       [("state", f32(N, 2, 64, 64).half(), TypeError), ("state", f32(N - 1, 2, 64, 64), ValueError),
        ("state", f32(N, 1, 64, 64), ValueError)]]
BAD += [(tm.shift_norm, NORM, *bad) for bad in
        [("x", rows(F32), TypeError), ("delta", rows(BF16), TypeError), ("delta", rows(t=1), ValueError),
         ("mu", f32(3, C).bfloat16(), TypeError), ("mu", f32(3, 64), ValueError), ("mu", f32(C), ValueError)] +
        [(q, z, e) for q in ("gamma", "beta") for z, e in ((f32(C).half(), TypeError), (f32(C).double(), TypeError),
                                                          (f32(64), ValueError), (f32(1, C), ValueError))] + BAD_CU +
        [("shift", rows(F32, t=N), TypeError), ("shift", rows(t=N + 1), ValueError), ("shift", rows(t=N, c=64), ValueError)]]
BAD += [(tm.head_gate, GATE, *bad) for bad in
        [(q, z, e) for q in "rkvg" for z, e in ((rows(F32), TypeError), (rows(BF16), TypeError), (rows(t=1), ValueError))] +
        [(q, z, e) for q in ("gamma", "beta", "u") for z, e in ((f32(C).bfloat16(), TypeError), (f32(64), ValueError),
                                                               (f32(2, 64), ValueError))]]


@pytest.mark.parametrize("fn,good,name,value,error", BAD, ids=["%s-%s-%d" % (b[0].__name__, b[2], i) for i, b in enumerate(BAD)])
def test_types_and_shapes(fn, good, name, value, error):
    with pytest.raises(error, match=name):
        fn(**dict(good, **{name: value}))


@pytest.mark.parametrize("width", [72, 96, 32])
def test_widths_of_broken_heads(width):
    """The columns past the last whole head would never be written."""
    x = rows(c=width)
    with pytest.raises(ValueError, match="heads"):
        tm.time_mix(x, x, x, x, x, x, CU)
    with pytest.raises(ValueError, match="heads"):
        tm.head_gate(x, x, x, x, x, f32(width), f32(width), f32(width))


@pytest.mark.parametrize("fn,good", [(tm.time_mix, MIX), (tm.shift_norm, NORM), (tm.head_gate, GATE)])
def test_tensors_elsewhere(fn, good):
    with pytest.raises(ValueError, match="GPU"):
        fn(**good)


SERVE = dict(x=rows(), delta=rows(), cu=CU, shift=rows(t=3), state=f32(3, 2, 64, 64), slots=torch.zeros(N, dtype=torch.int32))


@pytest.mark.parametrize("name,value,error", [
    ("x", rows(c=256), ValueError), ("x", rows(BF16), TypeError), ("delta", rows(t=1), ValueError), ("delta", rows(F32), TypeError),
    *BAD_CU, ("shift", rows(F32, t=3), TypeError), ("shift", rows(t=3, c=64), ValueError), ("state", f32(2, 2, 64, 64), ValueError),
    ("state", f32(3, 2, 64, 64).half(), TypeError), ("state", f32(3, 2, 64, 128)[..., ::2], ValueError),
    ("slots", torch.zeros(N, dtype=torch.int64), TypeError), ("slots", torch.zeros(1, dtype=torch.int32), ValueError)])
def test_serving(name, value, error):
    layer = tm.TimeMix(C, rank=8, device="cpu")
    layer.quantized = {}
    given = dict(SERVE, **{name: value})
    if name == "x":
        given["delta"] = None
    with pytest.raises(error, match=name):
        layer.serve(**given)
    with pytest.raises(ValueError, match="GPU"):
        layer.serve(**SERVE)


def test_serving_nothing(monkeypatch):
    """Empty sequences only: the products take no null addresses, which empty
    tensors have."""
    monkeypatch.setattr(tm, "_on_gpu", lambda *ts: None)
    layer = tm.TimeMix(C, rank=8, device="cpu")
    layer.quantized = {}
    shift, state = torch.ones(3, C, dtype=F16), torch.ones(3, 2, 64, 64)
    for delta in (None, rows(t=0)):
        full, out = layer.serve(rows(t=0), delta, tm.offsets([0, 0], "cpu"), shift, state, torch.zeros(2, dtype=torch.int32))
        assert full.shape == out.shape == (0, C) and out.dtype == F16
    assert bool((shift == 1).all()) and bool((state == 1).all())


def test_command_needs_prompts(capsys):
    """The row after an empty prompt would be another prompt's."""
    with pytest.raises(SystemExit):
        tm.main(["--prompts", "3,0"])
    assert "at least one token" in capsys.readouterr().err
