"""The delta rule's answers of bfloat16 rows where what the state gives and what the block's writes give cancel: A T enters as two
bfloat16 terms, and one would show.

In a block that starts from S, y = scale (e^gam Q S + (A T) R) with R = beta (V - e^gam K S). As in gdr_testlib.py variances add up: eta
of a product of computed operands, what A, T, R and A T carry, `few` for exponentials; six deviations are allowed."""

import numpy as np
import pytest
import torch

from gdr_testlib import deviations, forward
from operators_testlib import U, check, f64
from test_gdr_gpu import case, run

pytestmark = pytest.mark.gpu


def answers(q, k, v, g, beta, S, scale, eta):
    """The variances of a block's answers, A T and R."""
    few = (64 * U) ** 2
    b, gam = beta[:, None], np.cumsum(g)
    D = np.tril(np.exp(np.minimum(gam[:, None] - gam[None, :], 0.0)))
    eg = np.exp(gam)[:, None]
    G, A = np.tril(k @ k.T * D, -1), q @ k.T * D
    T = np.linalg.inv(np.eye(len(k)) + b * G)
    K2, Q2, S2, T2, D2, N2 = k ** 2, q ** 2, S ** 2, T ** 2, D ** 2, (b * G) ** 2
    vG, vA = np.tril(eta * D2 * (K2 @ K2.T) + few * G ** 2, -1), eta * D2 * (Q2 @ K2.T) + few * A ** 2
    vT = T2 @ (b ** 2 * vG) @ T2 + 6 * eta * (T2 + T2 @ N2 @ T2)
    R = b * (v - eg * (k @ S))
    vR = b ** 2 * eg ** 2 * (eta * (K2 @ S2)) + few * R ** 2
    AT2 = (A @ T) ** 2
    vAT = vA @ T2 + A ** 2 @ (vT + eta * T2) + eta * AT2
    return scale ** 2 * (eta * eg ** 2 * (Q2 @ S2) + few * eg ** 2 * (q @ S) ** 2 + AT2 @ vR + (vAT + eta * AT2) @ R ** 2), A @ T, R


def cancelling(dk, dv, Hv, n):
    """One row writes, with strength 1 and a key of nearly length 1, that there is nothing; the queries, multiples of that key, find what
    it leaves of the state."""
    c = case([n], Hk=Hv, Hv=Hv, dk=dk, dv=dv)
    c["q"].copy_(c["k"][:1].float() * torch.linspace(0.5, 1.0, n, device=c["k"].device)[:, None, None])
    c["v"].zero_()
    c["beta"].zero_()
    c["beta"][0] = 1.0
    c["g"].mul_(0.05)
    return c


@pytest.mark.parametrize("n", [64, 37])
@pytest.mark.parametrize("dk, dv, Hv", [(64, 64, 2), (128, 128, 3), (72, 40, 1), (64, 128, 80), (128, 128, 160)])
def test_answers_that_cancel(dk, dv, Hv, n):
    c = cancelling(dk, dv, Hv, n)
    y = run(c, False)["y"]
    want, tol, shown = expected(c)
    check("y", y, want, tol, y.dtype)
    assert shown > 0.3   # with a term less, that part of the answers would have been off by twice what is allowed


def expected(c):
    s, eta, shown = c["spec"], deviations("bf16")[0] ** 2, 0
    want, tol = np.zeros((s.rows, s.v_heads, s.dv)), np.zeros((s.rows, s.v_heads, s.dv))
    x = {m: f64(c[m]) for m in ("q", "k", "v", "g", "beta")}
    for h in range(s.v_heads):
        a = [x["q"][:, h], x["k"][:, h], x["v"][:, h], x["g"][:, h], x["beta"][:, h], f64(c["h0"])[0, h], s.scale]
        want[:, h] = forward(*a)[0]
        var, AT, R = answers(*a, eta)
        tol[:, h] = 6 * var ** 0.5
        once = torch.from_numpy(AT).float().bfloat16().double().numpy()
        shown += int((abs(s.scale * (once - AT) @ R) > 2 * (tol[:, h] + 2.0 ** -8 * (abs(want[:, h]) + tol[:, h]))).sum())
    return want, tol, shown / want.size
