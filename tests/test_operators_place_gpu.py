"""Tensors of another GPU than the current one, whose stream a call would use, are refused by name before any launch. One GPU
is enough: the tests tell the binding that another one is current."""

import pytest
import torch

import sparse_slot_memory_gb300 as sdm
from sparse_slot_memory_gb300 import operators

pytestmark = pytest.mark.gpu


def calls():
    rows, one = sdm.GlrSpec(P=1, rows=8, D=8, x_dtype="f32"), sdm.RopeSpec(8, 1, 1, 8, 8, 8, dtype="f32")
    x, h, t = (torch.zeros(8, 8, device="cuda") for _ in range(3))
    heads = lambda: torch.zeros(8, 1, 8, device="cuda")
    ids, row = torch.zeros(8, dtype=torch.int32, device="cuda"), torch.zeros(8, device="cuda")
    lp = sdm.LogprobSpec(rows=8, V=8, dtype="f32")
    return {
        "glr_forward": lambda: sdm.glr_forward(rows, x, x, h),
        "glr_backward": lambda: sdm.glr_backward(rows, x, x, x, sdm.alloc_glr_states(rows), h, t),
        "glr_step": lambda: sdm.glr_step(rows, x, x, h, t, slots=ids),
        "qk_norm_rope": lambda: sdm.qk_norm_rope(one, heads(), heads(), ids, t, None, None, heads(), heads()),
        "qk_norm_rope_backward": lambda: sdm.qk_norm_rope_backward(one, heads(), heads(), heads(), heads(), ids, t, None, None,
                                                                   heads(), heads()),
        "rope_table": lambda: sdm.rope_table(one, [1.0] * 4, t),
        "token_logprobs": lambda: sdm.token_logprobs(lp, x, ids, row),
        "token_logprobs_backward": lambda: sdm.token_logprobs_backward(lp, x, ids, row, row, row, h),
    }


@pytest.mark.parametrize("name", ["glr_forward", "glr_backward", "glr_step", "qk_norm_rope", "qk_norm_rope_backward",
                                  "rope_table", "token_logprobs", "token_logprobs_backward"])
def test_tensors_of_another_gpu_are_refused(name, monkeypatch):
    call = calls()[name]
    call()
    torch.cuda.synchronize()
    other = torch.cuda.current_device() + 1
    monkeypatch.setattr(operators, "_alone", False, raising=False)
    monkeypatch.setattr(operators, "_here", lambda: other, raising=False)
    with pytest.raises(ValueError, match=f"lies on GPU {other - 1}, the current one is GPU {other}"):
        call()


def test_one_gpu_needs_no_look(monkeypatch):
    """Where there is one GPU, no call asks where its tensors lie."""
    call = calls()["glr_step"]
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 1)
    call()
    spec = sdm.GlrSpec(P=1, rows=8, D=8, x_dtype="f32")
    spec.c()
    monkeypatch.setattr(operators, "_here", lambda: 1 / 0, raising=False)
    call()


def test_optional_arrays_too(monkeypatch):
    lp = sdm.LogprobSpec(rows=2, V=8, dtype="f32")
    x, ids, row = torch.zeros(2, 8, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, device="cuda")
    here = torch.cuda.current_device()

    class Elsewhere(torch.Tensor):
        """A view of memory of this GPU that says it is the next one's."""

        def get_device(self):
            return here + 1

    sdm.token_logprobs(lp, x, ids, row)
    monkeypatch.setattr(operators, "_alone", False, raising=False)
    entropy = row.clone().as_subclass(Elsewhere)
    with pytest.raises(ValueError, match="entropy: lies on GPU"):
        sdm.token_logprobs(lp, x, ids, row, entropy=entropy)
