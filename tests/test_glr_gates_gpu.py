"""The gates' exponential of the gated linear recurrence: its own error, and what a long memory makes of it."""

import math

import pytest
import torch

import sparse_slot_memory_gb300 as sdm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def gates(g):
    """exp(g) as the recurrence has it: a state of 1 and an input of 0."""
    n = g.numel() // 4
    g = g[:4 * n].view(n, 4)
    state, y = torch.ones(n, 4, device="cuda"), torch.empty(n, 4, device="cuda")
    sdm.glr_step(sdm.GlrSpec(P=1, rows=n, D=4, x_dtype="f32"), torch.zeros(n, 4, device="cuda"), g.contiguous(), state, y)
    return y.view(-1), g.reshape(-1).double().exp()


@pytest.mark.parametrize("low, high", [(1e-7, 1e-6), (1e-6, 1e-5), (1e-5, 1e-4), (1e-4, 1e-3), (1e-3, 1e-2), (1e-2, 0.1), (0.1, 1.0),
                                       (1.0, 10.0), (10.0, 80.0)])
def test_error_of_a_gate(low, high):
    """Within 4 u + 1.25 |g| u (2^t within 4 u; the product g log2(e) is rounded by u |g| of what it gives, and log2(e) to a
    float32 by 0.22 u); never above 1; where long memories lie, no more than a quarter of u off on average, half of what the
    rounding of a value below 1 to a float32 is at most."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    g = -torch.exp(torch.empty(1 << 20, device="cuda").uniform_(math.log(low), math.log(high), generator=gen))
    y, want = gates(g)
    err = (y.double() - want) / want
    assert bool((err.abs() <= (4 + 1.25 * g.abs()) * U).all()) and bool((y <= 1).all())
    if high <= 1.0:
        assert abs(float(err.mean())) <= 0.25 * U


def test_gates_that_are_exact():
    g = torch.tensor([0.0, -0.0, -1e-30, -1e-9, -float("inf"), torch.finfo(torch.float32).min, -1e30, 0.0], device="cuda")
    assert gates(g)[0].tolist() == [1, 1, 1, 1, 0, 0, 0, 1]


@pytest.mark.parametrize("gw", [1, 32])
@pytest.mark.parametrize("mean", [0.0, 3.0, 6.0, 9.0])
def test_long_memories_are_as_exact_as_row_by_row(mean, gw):
    """Over 3000 rows the error of float32 outputs is no more than a quarter above that of float32 rows computed one by one
    with exp rounded to float32."""
    T, P, D = 3000, 4, 256
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(P * T, D, device="cuda", generator=gen)
    g = torch.nn.functional.logsigmoid(torch.randn(P * T, D // gw, device="cuda", generator=gen) + mean)
    y = torch.empty_like(x)
    sdm.glr_forward(sdm.GlrSpec(P=P, rows=P * T, D=D, gate_width=gw, x_dtype="f32"), x, g, y)
    a, b = (v.repeat_interleave(gw, 1).view(P, T, D) for v in (g.double().exp(), g.exp()))
    x, y = x.view(P, T, D), y.view(P, T, D)
    h, one, mine, theirs = torch.zeros(P, D, dtype=torch.float64, device="cuda"), torch.zeros(P, D, device="cuda"), 0.0, 0.0
    for t in range(T):
        h = a[:, t] * h + x[:, t]
        one = b[:, t] * one + x[:, t]
        mine, theirs = mine + (y[:, t] - h).square().sum(), theirs + (one - h).square().sum()
    assert float((mine / theirs).sqrt()) <= 1.25
