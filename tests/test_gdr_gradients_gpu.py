"""The delta rule's gradients of bfloat16 queries and keys are as exact as their rounding: what enters the products before it has two
bfloat16 terms, 2^-17, so that beside the rounding's own error, about 2^-9 of a value, nothing is to be seen. Of the squares a few
products of 2^-17 bring (2^-6)^2; a hundredth is allowed. With one term the error is a quarter larger."""

import numpy as np
import pytest
import torch

from operators_testlib import f64
from test_gdr_float32_gpu import rule
from test_gdr_gpu import case, run

pytestmark = pytest.mark.gpu

CASES = {
    "d64": dict(lens=[500, 333], Hk=2, Hv=2, dk=64, dv=64), "d128": dict(lens=[400], Hk=2, Hv=2, dk=128, dv=128),
    "shared": dict(lens=[257, 64], Hk=1, Hv=4, dk=128, dv=64), "d72_56": dict(lens=[300, 41, 64], Hk=1, Hv=3, dk=72, dv=56),
    "slow": dict(lens=[600], dk=64, dv=128, rate=0.01), "units": dict(lens=[450, 64, 3], Hk=8, Hv=32, dk=64, dv=64),
    "alike": dict(lens=[300], Hk=2, Hv=2, dk=128, dv=128, alike=1.0),
}


@pytest.mark.parametrize("name", list(CASES))
def test_as_exact_as_their_rounding(name):
    c = case(**CASES[name])
    r = run(c)
    x = {n: f64(c[n]) for n in ("q", "k", "v", "g", "beta", "dy", "h0", "dhT")}
    want = rule(x, c["cuts"], c["spec"].scale, np.float64)
    for n in ("y", "dq", "dk", "dv"):
        rounded = torch.from_numpy(want[n]).to(torch.bfloat16).double().numpy()
        assert np.linalg.norm(f64(r[n]) - want[n]) <= 1.01 * np.linalg.norm(rounded - want[n]), n
