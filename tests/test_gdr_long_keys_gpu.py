"""Keys longer than 1: the matrix that a segment of a long sequence makes of the state before it may leave float32's range where the
states do not. The segment before then walks on, here the first one, so a sequence alone in its call has what it has beside others."""

import numpy as np
import pytest
import torch

import sparse_slot_memory_gb300 as sdm
from gdr_testlib import forward
from operators_testlib import U, check, f64
from test_gdr_gpu import case

pytestmark = pytest.mark.gpu

ROWS, HEADS = 4160, 2


def walk(c, beside, states=False):
    """The case's sequence alone, or the first of many in one call, whose walks are whole."""
    s, x = c["spec"], [c[n] for n in ("q", "k", "v", "g", "beta")]
    P = 1 + beside
    spec = sdm.GdrSpec(P=P, rows=s.rows, k_heads=s.k_heads, v_heads=s.v_heads, dk=s.dk, dv=s.dv, scale=s.scale)
    offsets = torch.full((P + 1,), s.rows, device="cuda")
    offsets[0] = 0
    h0 = torch.zeros(P, s.v_heads, s.dk, s.dv, device="cuda")
    h0[0] = c["h0"][0]
    y, hT, ws = torch.empty_like(c["v"]).fill_(float("nan")), torch.empty_like(h0), sdm.alloc_gdr_workspace(spec)
    ws.fill_(255)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sdm.gdr_forward(spec, *x, y, ws, offsets=offsets, h0=h0, hT=hT, status=st, states=sdm.alloc_gdr_states(spec) if states else None)
    assert int(st.item()) == 0
    return y, hT[:1]


def long_keys(kind, dk, Hk):
    """One value head (the last) of two with keys along the first channel, of strength 1. Of length 2 every row multiplies what the
    state has there by -3: the state has nothing there. Of length 3^1/2 by -2: the state starts anew every 150 rows, from values that
    are small enough."""
    c = case([ROWS], Hk=Hk, Hv=HEADS, dk=dk, dv=64)
    c["k"][:, -1] = 0.0
    c["beta"][:, -1] = 1.0
    if kind == "nothing there":
        c["k"][:, -1, 0] = 2.0
        c["v"][:, -1] = 0.0
        c["h0"][:, -1, 0] = 0.0
        c["g"][:, -1] = -2.0 ** -10
    else:
        c["k"][:, -1, 0] = 3.0 ** 0.5
        c["v"][:, -1] *= 2.0 ** -80
        c["h0"][:, -1] *= 2.0 ** -80
        c["g"][:, -1] = 0.0
        c["g"][::150, -1] = -float("inf")
    return c


@pytest.mark.parametrize("dk", [64, 72])
@pytest.mark.parametrize("kind", ["nothing there", "starts anew"])
def test_alone_as_beside_others(kind, dk):
    c = long_keys(kind, dk, HEADS)
    y, hT = walk(c, 0)
    # the other head as if this one's keys were short
    short = dict(c) | {"k": c["k"].clone()}
    short["k"][:, -1] *= 0.25
    ys, hs = walk(short, 0)
    assert torch.equal(y[:, 0], ys[:, 0]) and torch.equal(hT[:, 0], hs[:, 0])
    # 160 sequences of two heads are more walks than SMs: each is walked whole. Columns of 64 or fewer have the same sums
    yw, hw = walk(c, 159)
    assert bool(y.isfinite().all()) and bool(hT.isfinite().all())
    assert torch.equal(y[:, 1], yw[:, 1]) and torch.equal(hT[:, 1], hw[:, 1])
    a, b = walk(c, 0, states=True), walk(c, 0)
    assert all(torch.equal(m, n) for m, n in zip(a, b))


def test_value_heads_that_share_long_keys():
    c = long_keys("nothing there", 64, 1)
    c["v"].zero_()
    c["h0"][:, :, 0] = 0.0
    c["beta"].fill_(1.0)
    y, hT = walk(c, 0)
    yw, hw = walk(c, 159)
    assert bool(y.isfinite().all()) and torch.equal(y, yw) and torch.equal(hT, hw)


def test_a_state_that_has_nothing_where_the_keys_lie():
    """It decays by itself: per block of rows one rounding and the error of an exponential, 64 u; an answer's sum of dk products is 24
    2^-23 off beside that and its operand 2^-17."""
    c = long_keys("nothing there", 64, HEADS)
    y, hT = walk(c, 0)
    s, h = c["spec"], 1
    x = {n: f64(c[n])[:, h] for n in ("q", "k", "v", "g", "beta")}
    wy, states, _ = forward(x["q"], x["k"], x["v"], x["g"], x["beta"], f64(c["h0"])[0, h], s.scale)
    off = (ROWS // 64 + 1) * 65 * U
    mag = s.scale * np.stack([abs(states[t + 1]).T @ abs(x["q"][t]) for t in range(ROWS)])
    check("y", y[:, h], wy, (off + 2.0 ** -17 + 24 * 2.0 ** -23) * mag, torch.bfloat16)
    check("hT", hT[0, h], states[-1], off * abs(states[-1]))
