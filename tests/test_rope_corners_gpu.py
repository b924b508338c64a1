"""Corners of the norm and rotation of heads: the gradients of weights that are not used, padding tokens beside a table that is
not filled and weights that are not finite."""

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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("hd, rd, layout", [(64, 64, "half"), (120, 64, "interleaved"), (320, 320, "half"), (64, 0, "half")])
@pytest.mark.parametrize("norm", [True, False])
def test_padding_tokens_read_no_row_of_the_table(dtype, hd, rd, layout, norm):
    """A table may hold the rows of the positions in use alone: padding tokens take none of them. Their outputs and
    gradients are 0 also where a weight is infinite, and they add nothing to the weights' gradients."""
    T, max_pos = 20, 64
    q, k, dqo, dko = heads(T, 5, 1, hd, dtype)
    spec = sdm.RopeSpec(tokens=T, q_heads=5, k_heads=1, hd=hd, rot_dim=rd, max_pos=max_pos, layout=layout, norm=norm,
                        dtype="f32" if dtype == torch.float32 else "bf16")
    table = torch.full((max_pos, rd), float("nan"), device="cuda")
    table[30:60] = torch.randn(30, rd, device="cuda")
    pos = torch.arange(30, 30 + T, dtype=torch.int32, device="cuda")
    pad = torch.zeros(T, dtype=torch.bool, device="cuda")
    pad[[0, 3, 7, T - 1]] = True
    pos[pad] = torch.tensor([-1, -5, max_pos, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    w = 1 + 0.1 * torch.randn(hd, device="cuda")
    q[pad], dko[pad] = float("nan"), float("inf")   # nor are padding tokens' rows looked at

    def call(w):
        o = [torch.full_like(v, float("nan")) for v in (q, k, q, k)]
        dw = [torch.full((hd,), float("nan"), device="cuda") for _ in range(2)]
        sdm.qk_norm_rope(spec, q, k, pos, table, w, w, o[0], o[1])
        sdm.qk_norm_rope_backward(spec, dqo, dko, q, k, pos, table, w, w, o[2], o[3], *dw, sdm.alloc_rope_workspace(spec))
        return o, dw

    o, dw = call(w)
    for v in o:
        assert bool((v[pad] == 0).all()) and bool(torch.isfinite(v[~pad]).all())
    assert all(bool(torch.isfinite(v).all()) for v in dw)
    w[1] = float("inf")
    o, _ = call(w)
    for v in o:
        assert bool((v[pad] == 0).all())
