"""How the time-mixing functions stand in autograd, on the CPU: the library's
entries are replaced by stand-ins that fill their outputs."""

import pytest
import torch

from gemm_rwkv_amd import time_mix as tm

T, C, N = 4, 64, 1
CU = tm.offsets([T], "cpu")


def rows(n=T):
    return torch.ones(n, C, dtype=torch.float16, requires_grad=True)


def param(*shape):
    return torch.ones(*shape, requires_grad=True)


@pytest.fixture(autouse=True)
def library(monkeypatch):
    def fill(*args, **kw):
        for t in args:
            if isinstance(t, torch.Tensor) and t.is_floating_point() and not t.requires_grad:
                t.fill_(1)
    for name in ("rq_shift_norm", "rq_time_mix", "rq_head_gate"):
        monkeypatch.setattr(tm.rq, name, fill)
        monkeypatch.setattr(tm.rq, name + "_backward", fill)
    monkeypatch.setattr(tm, "_on_gpu", lambda *ts: None)


def outputs():
    return [("time_mix", tm.time_mix(*(rows() for _ in range(6)), CU, param(N, 1, 64, 64))),
            ("shift_norm", tm.shift_norm(rows(), rows(), param(2, C), param(C), param(C), CU, rows(N))),
            ("head_gate", (tm.head_gate(*(rows() for _ in range(5)), param(C), param(C), param(C)),))]


@pytest.mark.parametrize("i", range(3), ids=["time_mix", "shift_norm", "head_gate"])
def test_second_derivatives_are_refused(i):
    """The backward calls carry no graph: a derivative of theirs would silently
    lack these terms."""
    _, outs = outputs()[i]
    x = torch.ones((), requires_grad=True)
    loss = sum((o.float() * x * x).sum() for o in outs)
    inputs = [t for t, _ in outs[0].grad_fn.next_functions if hasattr(t, "variable")]
    leaf = inputs[0].variable
    grad, = torch.autograd.grad(loss, leaf, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        grad.float().sum().backward()


@pytest.mark.parametrize("i", range(3), ids=["time_mix", "shift_norm", "head_gate"])
def test_first_derivatives(i):
    _, outs = outputs()[i]
    leaves = [t.variable for t, _ in outs[0].grad_fn.next_functions if hasattr(t, "variable")]
    sum(o.float().sum() for o in outs).backward()
    assert len(leaves) >= 6
    for leaf in leaves:
        assert leaf.grad is not None and leaf.grad.shape == leaf.shape and leaf.grad.dtype == leaf.dtype
