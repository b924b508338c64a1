"""The gated delta rule in 64 bits, a row at a time, with the error that the kernels' arithmetic may have.

Roundings to nearest are independent of one another, so the errors that they leave add up like variances; a bound here is six
times the root of the sum of the variances (a part in 1e9 for one value, and the variances below are upper bounds). What
include/sdm.h states gives them, relative to the square root of sum a^2 b^2 for a product sum a b:
  * an operand of two bfloat16 terms is within 2^-17 (half a step of 8 bits, twice), a variance of at most 2^-34 / 3, and what
    a product of two such leaves out is below 2^-16, a variance of at most 2^-32 / 9; of three terms 2^-8 of these;
  * one bfloat16 term, which the answers take of A (and the gradients of queries and keys of their last products): 2^-8, 2^-16 / 3;
  * an addition of the tensor cores may cut off a unit in the last place, 2^-23 of the sum so far, 24 times in a row at most
    (192 summands, eight or sixteen at a time): 24 2^-23, which may all have one sign and is taken as a deviation; so are
    64 2^-24 for exponentials and the few products beside them.
Within a block of 64 rows the variances are followed through the block's formulas. Across blocks an error of the state is not
amplified: with keys no longer than 1 and strengths in [0, 1] every step S -> e^g (I - beta k k^T) S shortens each of its columns,
so the variances of a column's errors add up, and a row takes at most its own length times their root.
A sequence walked in segments (not `whole`) has each segment's matrix from walking the identity. Every block rounds its columns, no
longer than 1, as it rounds a state's: what the matrix then makes of the state before the segment is off by a variance of eta times
that state's squared lengths for every block (its writes' operands once, its state's once).
"""

from __future__ import annotations

import numpy as np

from operators_testlib import U

C = 64


def deviations(x_dtype):
    """Of a product of computed operands, of A in the answers, of the last products of the gradients of queries and keys."""
    cut, one = 24 * 2.0 ** -23, 2.0 ** -8 / 3 ** 0.5
    two = (2 * 2.0 ** -34 / 3 + 2.0 ** -32 / 9) ** 0.5
    return (two + cut, one, 2 ** 0.5 * one) if x_dtype == "bf16" else (two * 2.0 ** -8 + cut,) * 3


def forward(q, k, v, g, beta, S, scale):
    """Rows of one head: y, the state before every row and after the last, the errors v - e^g S^T k."""
    y, E, states = np.zeros_like(v), np.zeros_like(v), [S]
    for t in range(len(q)):
        S = np.exp(g[t]) * S
        E[t] = v[t] - S.T @ k[t]
        S = S + np.outer(k[t], beta[t] * E[t])
        y[t] = scale * (S.T @ q[t])
        states.append(S)
    return y, states, E


def backward(q, k, v, g, beta, states, E, scale, dy, dS):
    d = {"dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v), "dg": np.zeros_like(g), "dbeta": np.zeros_like(g)}
    behind = [None] * (len(q) + 1)   # the gradient of the state behind row t - 1, without what row t - 1's answer takes
    behind[len(q)] = dS
    for t in range(len(q) - 1, -1, -1):
        dS = dS + scale * np.outer(q[t], dy[t])
        before = np.exp(g[t]) * states[t]
        du = dS.T @ k[t]
        d["dq"][t] = scale * (states[t + 1] @ dy[t])
        d["dbeta"][t] = du @ E[t]
        d["dv"][t] = beta[t] * du
        d["dk"][t] = dS @ (beta[t] * E[t]) - before @ d["dv"][t]
        dS = dS - np.outer(k[t], d["dv"][t])
        d["dg"][t] = (dS * before).sum()
        dS = np.exp(g[t]) * dS
        behind[t] = dS
    return d, behind


def bounds(q, k, v, g, beta, states, E, scale, dy, behind, dev, whole=True):
    """The bounds of a head's outputs, block by block: forwards for the states, backwards for their gradients. v..: variances,
    ..2: squares."""
    n = len(q)
    eta, etaA, etag = (d * d for d in dev)
    few = (64 * U) ** 2
    t = {name: np.zeros_like(x) for name, x in (("y", v), ("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dbeta", g))}
    blocks = []
    vS = np.zeros(v.shape[1])   # of the columns of the state
    peak = np.zeros(v.shape[1])   # their largest squared lengths so far
    for r in range(0, n, C):
        s = slice(r, min(r + C, n))
        K, Q, V, S = k[s], q[s], v[s], states[r]
        b = np.maximum(beta[s], 2.0 ** -80)[:, None]
        gam = np.cumsum(np.maximum(g[s], -150.0))
        D = np.tril(np.exp(np.minimum(gam[:, None] - gam[None, :], 0.0)))
        eg, ec = np.exp(gam)[:, None], np.exp(gam[-1] - gam)[:, None]
        G, A = np.tril(K @ K.T * D, -1), Q @ K.T * D
        T = np.linalg.inv(np.eye(len(K)) + b * G)
        K2, Q2, S2, T2, D2, N2 = K ** 2, Q ** 2, S ** 2, T ** 2, D ** 2, (b * G) ** 2
        vG, vA = np.tril(eta * D2 * (K2 @ K2.T) + few * G ** 2, -1), eta * D2 * (Q2 @ K2.T) + few * A ** 2
        vT = T2 @ (b ** 2 * vG) @ T2 + 6 * eta * (T2 + T2 @ N2 @ T2)
        R = b * (V - eg * (K @ S))
        vR = b ** 2 * eg ** 2 * (eta * (K2 @ S2)) + few * R ** 2
        u = b * E[s]
        vU = T2 @ vR + (vT + eta * T2) @ R ** 2
        nq, nk = (Q2.sum(1) ** 0.5)[:, None], (K2.sum(1) ** 0.5)[:, None]
        t["y"][s] = scale ** 2 * (eta * eg ** 2 * (Q2 @ S2) + (vA + (eta + etaA) * A ** 2) @ u ** 2 + A ** 2 @ vU + nq ** 2 * vS)
        blocks.append(dict(s=s, S=S, S2=S2, K=K, Q=Q, K2=K2, Q2=Q2, nk=nk, nq=nq, b=b, D=D, eg=eg, ec=ec, G=G, A=A, vG=vG, vA=vA, T=T, vT=vT,
                           u=u, vU=vU, vS=vS))
        vS = vS + (K2.T @ (ec ** 2 * (vU + eta * u ** 2)) + eta * states[s.stop] ** 2).sum(0)
        peak = np.maximum(peak, S2.sum(0))
        if not whole:
            vS = vS + 2 * eta * peak
    t["hT"] = vS[None, :] + np.zeros_like(states[0])
    if dy is not None:
        vD = np.zeros(v.shape[1])
        for B in reversed(blocks):
            s, S2, K, K2, Q, Q2, nk, nq, b, D, eg, ec, G, A, vG, vA, T, vT, u, vS = (
                B[x] for x in ("s", "S2", "K", "K2", "Q", "Q2", "nk", "nq", "b", "D", "eg", "ec", "G", "A", "vG", "vA", "T", "vT", "u", "vS"))
            Y, dS = dy[s], behind[s.stop]
            Y2, dS2, T2, u2, D2, L2 = Y ** 2, dS ** 2, T ** 2, u ** 2, D ** 2, np.tril(D, -1) ** 2
            X = scale * A.T @ Y + ec * (K @ dS)
            vX = scale ** 2 * ((vA + eta * A ** 2).T @ Y2) + ec ** 2 * eta * (K2 @ dS2) + few * X ** 2
            W = T.T @ X
            vWl = T2.T @ vX + (vT + eta * T2).T @ X ** 2            # of the block's own
            W2, vW, vU = W ** 2, vWl + nk ** 2 * vD, B["vU"] + b ** 2 * nk ** 2 * vS
            t["dv"][s] = beta[s][:, None] ** 2 * vW
            M2, N2 = (b * (W @ u.T)) ** 2, (scale * Y @ u.T) ** 2
            vM = b ** 2 * (eta * W2 @ u2.T + vW @ u2.T + W2 @ vU.T)
            vN = scale ** 2 * (eta * Y2 @ u2.T + Y2 @ vU.T)
            vE = B["vU"] / b ** 2 + nk ** 2 * vS
            t["dbeta"][s] = (vW * E[s] ** 2 + W2 * vE + eta * W2 * E[s] ** 2).sum(1)
            sc = scale * eg
            ND, vND, MD, vMD = N2 * D2, vN * D2, M2 * L2, vM * L2
            e = etag + few
            t["dq"][s] = sc ** 2 * (eta * Y2 @ S2.T + (Y2 @ vS)[:, None]) + (vND + e * ND) @ K2
            t["dk"][s] = ((vND + e * ND).T @ Q2 + (vMD + e * MD) @ K2 + (vMD + e * MD).T @ K2
                          + (eg * b) ** 2 * (vW @ S2.T + (W2 @ vS)[:, None] + etag * (W2 @ S2.T))
                          + ec ** 2 * (vU @ dS2.T + (u2 @ vD)[:, None] + eta * u2 @ dS2.T))
            # the errors of a rectangle's terms share their causes: their deviations are added
            Z = np.tril((vN * A ** 2 + N2 * (vA + eta * A ** 2) + vM * G ** 2 + M2 * (vG + eta * G ** 2)) ** 0.5, -1)
            QS2, KS2, KD2 = (Q @ B["S"]) ** 2, (K @ B["S"]) ** 2, (K @ dS) ** 2
            a_ = (sc[:, 0] ** 2 * (Y2 * (eta * (Q2 @ S2) + nq ** 2 * vS + few * QS2)).sum(1)
                  + (eg * b)[:, 0] ** 2 * (vW * KS2 + W2 * (eta * (K2 @ S2) + nk ** 2 * vS + few * KS2)).sum(1)) ** 0.5
            e_ = (ec[:, 0] ** 2 * (vU * KD2 + u2 * (eta * (K2 @ dS2) + nk ** 2 * vD + few * KD2)).sum(1)) ** 0.5
            inner = eg[-1, 0] * ((vD * S2.sum(0) + vS * dS2.sum(0) + vD * vS).sum() + eta * (dS2 * S2).sum()) ** 0.5
            suffix = np.cumsum(Z[::-1], 0)[::-1]
            for i in range(len(K)):
                t["dg"][s.start + i] = (suffix[i, :i].sum() + a_[i:].sum() + e_[:i].sum() + inner) ** 2
            new = behind[s.start]
            vD = vD + (Q2.T @ (sc ** 2 * eta * Y2) + K2.T @ ((eg * b) ** 2 * (vWl + eta * W2)) + eta * (new ** 2 + eg[-1] ** 2 * dS2)).sum(0)
        t["dh0"] = vD[None, :] + np.zeros_like(states[0])
    return {name: 6 * x ** 0.5 for name, x in t.items()}


def oracle(x, cuts, scale, x_dtype, train=True, whole=True):
    """x: float64 arrays q, k [rows, Hk, dk], v [rows, Hv, dv], g, beta [rows, Hv], h0 [P, Hv, dk, dv] (dy, dhT): the outputs'
    values and bounds, as the calls lay them out; rows of no sequence NaN."""
    Hk, Hv = x["k"].shape[1], x["v"].shape[1]
    R = Hv // Hk
    dev = deviations(x_dtype)
    names = {"y": "v", "hT": "h0"} | ({"dq": "q", "dk": "k", "dv": "v", "dg": "g", "dbeta": "g", "dh0": "h0"} if train else {})
    # a strength below 2^-80 counts as 2^-80
    x = x | {"beta": np.where(np.abs(x["beta"]) < 2.0 ** -80, np.copysign(2.0 ** -80, x["beta"]), x["beta"])}
    val = {n: np.full_like(x[m], np.nan) for n, m in names.items()}
    tol = {n: np.zeros_like(x[m]) for n, m in names.items()}
    for n in ("dq", "dk"):
        if train:
            for p in range(len(cuts) - 1):
                val[n][cuts[p]:cuts[p + 1]] = 0.0
    for p in range(len(cuts) - 1):
        s = slice(cuts[p], cuts[p + 1])
        for h in range(Hv):
            a = [x["q"][s, h // R], x["k"][s, h // R], x["v"][s, h], x["g"][s, h], x["beta"][s, h]]
            y, states, E = forward(*a, x["h0"][p, h], scale)
            val["y"][s, h], val["hT"][p, h] = y, states[-1]
            d, behind, dy = {}, None, None
            if train:
                dy = x["dy"][s, h]
                d, behind = backward(*a, states, E, scale, dy, x["dhT"][p, h])
                val["dh0"][p, h] = behind[0]
            b = bounds(*a, states, E, scale, dy, behind, dev, whole)
            tol["y"][s, h], tol["hT"][p, h] = b["y"], b["hT"]
            if train:
                tol["dh0"][p, h] = b["dh0"]
                for n in ("dv", "dg", "dbeta"):
                    val[n][s, h], tol[n][s, h] = d[n], b[n]
                for n in ("dq", "dk"):
                    val[n][s, h // R] += d[n]
                    tol[n][s, h // R] += b[n] + R * U * abs(d[n])
    return val, tol
