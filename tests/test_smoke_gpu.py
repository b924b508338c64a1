"""The smoke run of the operators: its GPU work is the operators' and little else, so that a list of its first launches shows
every one of them."""

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import __graft_entry__

pytestmark = pytest.mark.gpu


class CudaOps(TorchDispatchMode):
    """Counts torch's operations with a CUDA tensor among their results."""

    count = 0

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        flat = out if isinstance(out, (tuple, list)) else (out,)
        self.count += any(isinstance(t, torch.Tensor) and t.is_cuda for t in flat)
        return out


def test_the_operators_smoke_leaves_torch_little_to_launch():
    with CudaOps() as ops:
        __graft_entry__._smoke_operators()
    assert ops.count < 150, ops.count
