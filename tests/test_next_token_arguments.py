"""What the torch functions of a model's end refuse before the library is
called, which takes bare addresses.  Nothing runs on a GPU here: the library's
entries are stand-ins that fail the test when they are reached."""

import pytest
import torch

from gemm_rwkv_amd import next_token as nx, rq

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
M, C, N = 5, 256, 24
B128 = rq.RQ_FP8_E4M3_B128


@pytest.fixture(autouse=True)
def library(monkeypatch):
    for name in ("rq_norm_quantize", "rq_gemm_fp8_block", "rq_sample"):
        def reached(*args, _name=name, **kw):
            pytest.fail(_name + " was reached")
        monkeypatch.setattr(nx.rq, name, reached)


def rows(dtype=F16, m=M, c=C):
    return torch.zeros(m, c, dtype=dtype)


def weight(fmt=B128, k=C):
    return rq.QWeight(fmt, 0, N, k, torch.zeros(N * k, dtype=torch.uint8), torch.zeros(4, dtype=torch.uint8))


def codes(m=M, c=C, dtype=torch.uint8):
    return torch.zeros(m, c, dtype=dtype)


NORM = dict(x=rows(), delta=rows(), gamma=torch.zeros(C), beta=torch.zeros(C))
PRODUCT = dict(codes=codes(), scales=codes(c=4), w=weight())
SAMPLE = dict(logits=rows(F32), temperature=torch.ones(M), top_k=torch.ones(M, dtype=torch.int32), top_p=torch.ones(M),
              min_p=torch.ones(M), u=torch.ones(M))

BAD = [(nx.norm_quantize, NORM, *bad) for bad in
       [("x", rows(F32), TypeError), ("x", rows()[0], ValueError), ("delta", rows(BF16), TypeError), ("delta", rows(m=1), ValueError),
        ("norm", "layers", ValueError)] + [("fmt", fmt, ValueError) for fmt in (rq.RQ_F16, rq.RQ_W4_SYM, 77)] +
       [(q, z, e) for q in ("gamma", "beta")
        for z, e in ((torch.zeros(C).half(), TypeError), (torch.zeros(128), ValueError), (torch.zeros(1, C), ValueError))]]
BAD += [(nx.block_product, PRODUCT, *bad) for bad in
        [("codes", codes(dtype=torch.int8), TypeError), ("codes", codes(c=128), ValueError), ("codes", codes()[0], ValueError),
         ("scales", codes(c=2), ValueError), ("scales", codes(m=4, c=4), ValueError), ("scales", torch.zeros(M), TypeError),
         ("w", weight(rq.RQ_FP8_E4M3_CH), ValueError), ("dtype", torch.float64, TypeError)]]
BAD += [(nx.sample, SAMPLE, *bad) for bad in
        [("logits", rows(torch.float64), TypeError), ("logits", rows()[0], ValueError), ("logits", rows()[:, :0], ValueError),
         ("top_k", torch.ones(M), TypeError), ("top_k", torch.ones(M, dtype=torch.int64), TypeError),
         ("top_k", torch.ones(1, dtype=torch.int32), ValueError)] +
        [(q, z, e) for q in ("temperature", "top_p", "min_p", "u")
         for z, e in ((torch.ones(M).half(), TypeError), (torch.ones(M + 1), ValueError), (torch.ones(M, 1), ValueError),
                      (torch.tensor(1.0), ValueError))]]


@pytest.mark.parametrize("fn,good,name,value,error", BAD, ids=["%s-%s-%d" % (b[0].__name__, b[2], i) for i, b in enumerate(BAD)])
def test_types_and_shapes(fn, good, name, value, error):
    with pytest.raises(error, match="format" if name == "fmt" else name):
        fn(**dict(good, **{name: value}))


@pytest.mark.parametrize("fn,good", [(nx.norm_quantize, NORM), (nx.block_product, PRODUCT), (nx.sample, SAMPLE)])
def test_tensors_elsewhere(fn, good, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="current GPU"):
        fn(**good)


def test_no_gradient():
    with pytest.raises(RuntimeError, match="gradient"):
        nx.norm_quantize(rows().requires_grad_())
    with pytest.raises(RuntimeError, match="gradient"):
        nx.sample(rows(F32).requires_grad_())


def test_head():
    with pytest.raises(ValueError, match="128"):
        nx.Head(192, 100, device="cpu")
    with pytest.raises(ValueError, match="norm"):
        nx.Head(128, 100, norm="rms2", device="cpu")
    head = nx.Head(128, 100, device="cpu")
    with pytest.raises(RuntimeError, match="quantize"):
        head.next(rows(c=128))


def test_command_refuses_empty_prompts(capsys):
    with pytest.raises(SystemExit):
        nx.main(["--prompts", "3,0"])
    assert "at least one token" in capsys.readouterr().err
