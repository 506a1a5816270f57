"""Refusals of the time-mixing layer that need no GPU."""

import pytest
import torch

from gemm_rwkv_amd import time_mix as tm


def test_width_of_whole_groups():
    with pytest.raises(ValueError):
        tm.TimeMix(192, device="cpu")


def test_serving_needs_codes_and_float16():
    for dtype, error in ((torch.float16, RuntimeError), (torch.bfloat16, TypeError)):
        layer = tm.TimeMix(128, rank=8, dtype=dtype, device="cpu")
        if error is TypeError:
            layer.quantized = {}
        x = torch.zeros(1, 128, dtype=dtype)
        shift, state = layer.states(1)
        with pytest.raises(error):
            layer.serve(x, None, tm.offsets([1], "cpu"), shift, state, None)


def test_rows_of_other_types():
    x = torch.zeros(2, 64)
    with pytest.raises(TypeError):
        tm.time_mix(x, x, x, x, x, x, tm.offsets([2], "cpu"))


def test_offsets():
    assert tm.offsets([3, 0, 2], "cpu").tolist() == [0, 3, 3, 5]
