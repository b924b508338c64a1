"""Gates of the block's norm beside bfloat16 rows at their ends, forward and backward. The hardware's exponential and reciprocal are
off by 2^-21 (|z| + 1) of the value; where sigmoid(z) or what it leaves of 1 is below 2^-126 it is 0, so z sigmoid(z) and the
slopes, which take up to 88 of it, are off by 2^-119 at most, and have their limits where |z| is 88 or more."""

import numpy as np
import pytest
import torch

from operators_testlib import check, f64
from test_block_norm_gpu import EPS, act_of, case, oracle, run

pytestmark = pytest.mark.gpu

INF = float("inf")
ENDS = [-INF, -3e38, -1000.0, -104.0, -90.0, -88.5, -87.5, -86.0, -81.0, -80.0, -40.0, 0.0, 40.0, 80.0, 81.0, 86.0, 87.5, 88.5, 90.0, 104.0, 1000.0]


def compare(s, c, r):
    """The bounds of float32 rows' gates, and beside them what the gates may be off (rows that are not normed behind the sum)."""
    val, tol = oracle(c, f64(r["r"]), s)
    x = {n: f64(v) for n, v in c.items() if isinstance(v, torch.Tensor)}
    o, z, dr = x["o"], x["z"], x["dr"]
    p = 1 / np.sqrt((o ** 2).mean(1, keepdims=True) + EPS) if s.post else 1.0
    h, w, cs = o * p, x.get("w_post", 1.0), x.get("cs", 1.0)
    act, slope, mag = act_of(s.gate, z)
    rel = 2.0 ** -21 * (np.minimum(abs(z), 104.0) + 1)
    off, bend = rel * abs(act) + 2.0 ** -119, 2 * rel * mag + 2.0 ** -119
    dn = s.scale * cs * dr
    v = abs(dn * w) * off
    more = {"r": abs(s.scale * cs * h * w) * off, "dz": abs(dn * h * w) * bend, "dcs": (abs(s.scale * dr * h * w) * off).sum(0),
            "dw_post": (abs(dn * h) * off).sum(0), "do": p * (v + abs(o) * p * p * (v * abs(o)).mean(1, keepdims=True)) if s.post else v}
    for n in r:
        check(n, r[n], val[n], tol[n] + more.get(n, 0.0), torch.float32 if n in ("dw_post", "dcs") else torch.bfloat16)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", ["sigmoid", "silu"])
def test_ends(gate, post):
    ends = ENDS + [3e38, INF] if gate == "sigmoid" else ENDS   # z itself is beyond the rows' type with a weight above 1
    s, c = case(7, 4 * len(ends), gate=gate, pre=False, post=post)
    c["z"][:] = torch.tensor(ends, device="cuda").repeat(4)
    compare(s, c, run(s, c))


@pytest.mark.parametrize("gate", ["sigmoid", "silu"])
def test_limits_without_a_stream(gate):
    """A closed gate leaves nothing of the block's output and passes nothing back, also where nothing is added."""
    s, c = case(5, 64, gate=gate, pre=False, res=False)
    for z in (-INF, -3e38, -200.0, -88.0):
        c["z"].fill_(z)
        r = run(s, c)
        assert all(bool((r[n] == 0).all()) for n in ("r", "do", "dz", "dw_post", "dcs")), z
    c["z"].fill_(88.0)
    r = run(s, c)
    if gate == "sigmoid":
        assert bool((r["dz"] == 0).all())


@pytest.mark.parametrize("gate", ["sigmoid", "silu"])
def test_a_gate_that_is_not_a_number_stays_in_its_row(gate):
    s, c = case(40, 132, gate=gate, pre=False)
    clean = run(s, c)
    c["z"][7, 3] = float("nan")
    r = run(s, c)
    rows = [i for i in range(40) if i != 7]
    for n in ("r", "do", "dz"):
        assert torch.equal(r[n][rows], clean[n][rows]), n
        assert bool(r[n][7, 3].isnan()), n
    assert int(r["r"].isnan().sum()) == 1 and int(r["dz"].isnan().sum()) == 1
