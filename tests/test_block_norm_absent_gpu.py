"""Gradients of weights that a shape does not have (sdm_block_norm_backward): asked for, they are zeros, whatever the workspace
holds, and beside them the others are what they are alone."""

import pytest
import torch

import sparse_slot_memory_gb300 as sdm
from test_block_norm_gpu import case, run

pytestmark = pytest.mark.gpu


def backward(s, c, r, ws, **grads):
    o = torch.empty_like(c["o"])
    sdm.block_norm_backward(s, c["o"], r, c.get("dr"), o, ws, z=c.get("z"), dy=c.get("dy"), w_post=c.get("w_post"), w_pre=c.get("w_pre"),
                            channel_scale=c.get("cs"), dz=torch.empty_like(o) if s.gate != "none" else None, **grads)
    return o


def nan(n):
    return torch.full((n,), float("nan"), device="cuda")


SHAPES = {
    "no_post": dict(rows=50, D=260, post=False), "no_post_groups": dict(rows=9, D=512, group=128, post=False, xt="f32"),
    "no_pre": dict(rows=700, D=132, pre=False, gate="silu"), "neither": dict(rows=33, D=64, post=False, pre=False, xt="f32"),
    "one_row": dict(rows=1, D=4, post=False, pre=False), "wide": dict(rows=5, D=16384, pre=False),
}


@pytest.mark.parametrize("name", list(SHAPES))
def test_zeros_beside_the_others(name):
    s, c = case(**SHAPES[name])
    want = run(s, c)
    g = {"dw_post": nan(s.group or s.D), "dw_pre": nan(s.D), "d_channel_scale": nan(s.D)}
    ws = sdm.alloc_block_norm_workspace(s)
    ws.fill_(255)
    o = backward(s, c, want["r"], ws, **g)
    assert torch.equal(o, want["do"]) and torch.equal(g["d_channel_scale"], want["dcs"])
    for n, there in (("dw_post", s.post), ("dw_pre", s.pre)):
        assert torch.equal(g[n], want[n]) if there else bool((g[n] == 0).all()), n


@pytest.mark.parametrize("name", list(SHAPES))
def test_zeros_alone_need_no_workspace(name):
    s, c = case(**SHAPES[name])
    want = run(s, c, train=False)
    g = {}
    if not s.post:
        g["dw_post"] = nan(s.group or s.D)
    if not s.pre:
        g["dw_pre"] = nan(s.D)
    backward(s, c, want["r"], None, **g)
    assert all(bool((t == 0).all()) for t in g.values())
