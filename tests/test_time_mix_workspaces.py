"""Which workspaces the time-mixing layer's calls get, on the CPU with
stand-ins for the library's entries: calls that may run at the same time may
not share one."""

import pytest
import torch

from gemm_rwkv_amd import time_mix as tm

T, C = 4, 128
CU = tm.offsets([T], "cpu")
WITH = ("rq_time_mix", "rq_shift_norm_backward", "rq_head_gate_backward", "rq_fused_rkv", "rq_gemm_small_m", "rq_gemm_w4")


@pytest.fixture()
def given(monkeypatch):
    """(entry, its ws argument) of every call that takes one."""
    got = []
    for name in WITH + ("rq_shift_norm", "rq_head_gate", "rq_time_mix_backward"):
        def stand_in(*args, _name=name, **kw):
            if _name in WITH:
                got.append((_name, kw.get("ws")))
            for t in args:
                if isinstance(t, torch.Tensor) and t.is_floating_point() and not t.requires_grad:
                    t.fill_(1)
            return args[4] if _name.startswith("rq_gemm") else None
        monkeypatch.setattr(tm.rq, name, stand_in)
    monkeypatch.setattr(tm, "_on_gpu", lambda *ts: None, raising=False)
    return got


def rows():
    return torch.ones(T, C, dtype=torch.float16, requires_grad=True)


def test_every_torch_call_has_its_own(given):
    """None stands for the binding's workspace, which all such calls share."""
    param = lambda *s: torch.ones(*s, requires_grad=True)
    for _ in range(2):
        y, _ = tm.time_mix(*(rows() for _ in range(6)), CU)
        _, mixes, _ = tm.shift_norm(rows(), None, param(2, C), param(C), param(C), CU)
        gate = tm.head_gate(*(rows() for _ in range(5)), param(C), param(C), param(C))
        sum(o.float().sum() for o in (y, mixes, gate)).backward()
    assert sorted(n for n, _ in given) == sorted(WITH[:3] * 2)
    for name, ws in given:
        assert isinstance(ws, torch.Tensor) and ws.numel() == tm.rq.rq_workspace_bytes(), name
    assert len({id(ws) for _, ws in given}) == len(given)


@pytest.mark.parametrize("tokens", [1, 40])
def test_serving_passes_its_own_on(given, tokens):
    layer = tm.TimeMix(C, rank=8, device="cpu")
    layer.quantized = dict.fromkeys("rkvo")
    x = torch.zeros(tokens, C, dtype=torch.float16)
    shift, state = layer.states(1)
    ws = torch.zeros(16, dtype=torch.uint8)
    layer.serve(x, None, tm.offsets([tokens], "cpu"), shift, state, None, ws=ws)
    assert {n for n, _ in given} == {"rq_time_mix"} | ({"rq_fused_rkv", "rq_gemm_small_m"} if tokens <= 32 else {"rq_gemm_w4"})
    assert all(w is ws for _, w in given)
