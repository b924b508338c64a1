"""The delta rule of float32 rows is as exact as the rule in float32, a row at a time: its outputs' errors, in the root of their
squares, against those of the same rule in numpy's float32, both against 64 bits. A step of 16 summands may be cut off by a unit in
the last place where float32 rounds by half of one, which is twice a rounding's deviation; cut-offs have one sign, so those of the
four products that follow one another in a block (R, U, answers or gradients, states) add up like 4, not 2: 4 times the error."""

import numpy as np
import pytest

from gdr_testlib import backward, forward
from operators_testlib import f64
from test_gdr_gpu import case, run

pytestmark = pytest.mark.gpu

CASES = {
    "d64": dict(lens=[500, 333], Hk=2, Hv=2, dk=64, dv=64), "d128": dict(lens=[400], Hk=1, Hv=2, dk=128, dv=128),
    "d72_56": dict(lens=[300, 41, 64], Hk=1, Hv=3, dk=72, dv=56), "d24": dict(lens=[700], dk=24, dv=40), "slow": dict(lens=[600], dk=64, dv=64, rate=0.01),
    "alike": dict(lens=[300], dk=64, dv=64, alike=1.0), "wide": dict(lens=[200], dk=32, dv=128, Hv=2, rate=2.0),
}


def rule(x, cuts, scale, dtype):
    """Every output by the rule row by row in one type."""
    x = {n: t.astype(dtype) for n, t in x.items()}
    scale = dtype(scale)
    R = x["v"].shape[1] // x["k"].shape[1]
    d = {n: np.zeros_like(x[m]) for n, m in (("y", "v"), ("hT", "h0"), ("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"), ("dbeta", "g"), ("dh0", "h0"))}
    for p in range(len(cuts) - 1):
        s = slice(cuts[p], cuts[p + 1])
        for h in range(x["v"].shape[1]):
            a = [x["q"][s, h // R], x["k"][s, h // R], x["v"][s, h], x["g"][s, h], x["beta"][s, h]]
            y, states, E = forward(*a, x["h0"][p, h], scale)
            g, behind = backward(*a, states, E, scale, x["dy"][s, h], x["dhT"][p, h])
            d["y"][s, h], d["hT"][p, h], d["dh0"][p, h] = y, states[-1], behind[0]
            for n in ("dv", "dg", "dbeta"):
                d[n][s, h] = g[n]
            for n in ("dq", "dk"):
                d[n][s, h // R] += g[n]
    return d


@pytest.mark.parametrize("name", list(CASES))
def test_as_exact_as_float32(name):
    c = case(xt="f32", **CASES[name])
    r = run(c)
    x = {n: f64(c[n]) for n in ("q", "k", "v", "g", "beta", "dy", "h0", "dhT")}
    want, single = rule(x, c["cuts"], c["spec"].scale, np.float64), rule(x, c["cuts"], c["spec"].scale, np.float32)
    assert all(t.dtype == np.float32 for t in single.values())
    size = np.linalg.norm
    for n in r:
        assert size(f64(r[n]) - want[n]) <= 4 * size(single[n].astype(np.float64) - want[n]), n
