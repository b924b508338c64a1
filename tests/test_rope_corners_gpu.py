"""Corners of the norm and rotation of heads: the gradients of weights that are not used."""

import pytest
import torch

import sparse_slot_memory_gb300 as sdm

pytestmark = pytest.mark.gpu


def heads(T, Hq, Hk, hd, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    return [torch.randn(T, H, hd, generator=gen).to(dtype).cuda() for H in (Hq, Hk, Hq, Hk)]


@pytest.mark.parametrize("Hk", [2, 0])
def test_weight_gradients_without_the_norm_are_zero(Hk):
    """The rotation alone does not use the weights: their gradients are 0, and need no workspace."""
    q, k, dqo, dko = heads(33, 3, Hk, 64, torch.float32)
    spec = sdm.RopeSpec(tokens=33, q_heads=3, k_heads=Hk, hd=64, rot_dim=64, max_pos=40, dtype="f32", norm=False)
    table = torch.randn(40, 64, device="cuda")
    pos = torch.arange(33, dtype=torch.int32, device="cuda")
    w = torch.ones(64, device="cuda")
    dwq, dwk = (torch.full((64,), float("nan"), device="cuda") for _ in range(2))
    sdm.qk_norm_rope_backward(spec, dqo, dko, q, k, pos, table, w, w, torch.empty_like(q), torch.empty_like(k), dwq, dwk)
    assert bool((dwq == 0).all()) and bool((dwk == 0).all())
    dwk.fill_(float("nan"))
    sdm.qk_norm_rope_backward(spec, dqo, dko, q, k, pos, table, w, w, torch.empty_like(q), torch.empty_like(k), None, dwk)
    assert bool((dwk == 0).all())
