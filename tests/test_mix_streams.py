"""Where the memory of a state gradient's call comes from, on the CPU with a
stand-in for the allocator: one pool per stream, whose blocks are free for the
next call on that stream, in its order, and for no other."""

import contextlib

import pytest
import torch

import gemm_rwkv_amd.rq as rq

CURRENT, SIDE = 0, 7001


class Handle:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture()
def pools(monkeypatch):
    """The stream whose pool each allocation came from."""
    taken, now = [], [CURRENT]

    @contextlib.contextmanager
    def on(stream):
        now.append(stream.cuda_stream)
        yield
        now.pop()

    class Block:
        def data_ptr(self):
            return 1 << 20

        def record_stream(self, stream):
            pass

    def empty(n, dtype, device):
        taken.append((now[-1], n))
        return Block()

    monkeypatch.setattr(rq, "_gpu", lambda: True)
    monkeypatch.setattr(rq.torch, "empty", empty)
    monkeypatch.setattr(rq.torch.cuda, "stream", on)
    monkeypatch.setattr(rq.torch.cuda, "ExternalStream", Handle)
    monkeypatch.setattr(rq.torch.cuda, "default_stream", lambda: Handle(CURRENT))
    return taken


@pytest.mark.parametrize("stream,pool", [(None, CURRENT), (SIDE, SIDE), (Handle(SIDE), SIDE), (0, CURRENT)],
                         ids=["current", "handle", "stream", "null"])
def test_workspace_of_the_launch_stream(pools, stream, pool):
    p, n, keep = rq._fresh_ws(None, 4096, stream)
    assert pools == [(pool, 4096)] and p == keep.data_ptr() and n == 4096
