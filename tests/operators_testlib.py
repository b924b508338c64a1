"""The operators around the memory in 64 bits, written as loops and dense formulas, with the error that a float32
evaluation may have (u = 2^-24, half a unit in the last place of float32).

Every bound is derived from the arithmetic that include/sdm.h states, for any order of the sums:
  * expf, log2f, rsqrtf and the hardware's 2^t are within 2 ulp (4 u relative) of the exact value, + - * fma within u;
  * a sum of n terms in any order is within n u of the sum of their magnitudes;
  * a result stored in bfloat16 has one more relative rounding of 2^-8 (a unit in the last place of 8 bits, twice
    what round-to-nearest needs).
"""

from __future__ import annotations

import math

import numpy as np
import torch

U = 2.0 ** -24


def stored(dtype, value, tol):
    """The bound of a result after its rounding to `dtype`."""
    if dtype == torch.float32:
        return tol + 1e-37
    return tol + 2.0 ** -8 * (np.abs(value) + tol) + 1e-37


def check(name, got, want, tol, dtype=torch.float32):
    """got (a tensor of `dtype`) within tol of want; infinities and NaN in the same places."""
    assert got.dtype == dtype, (name, got.dtype)
    g = got.detach().double().cpu().numpy().reshape(np.shape(want))
    want = np.asarray(want, np.float64)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(g), np.isnan(want)), f"{name}: NaN in other places"
    assert np.array_equal(g[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), f"{name}: infinities"
    lim = np.broadcast_to(stored(dtype, want, tol), want.shape)
    bad = fine & ~(np.abs(g - np.where(fine, want, 0.0)) <= lim)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{name}: {bad.sum()} of {bad.size} off, first at {i}: {g[i]!r}, not {want[i]!r} +- {lim[i]!r}")


def f64(t):
    return t.detach().double().cpu().numpy()


# ---- gated linear recurrence -------------------------------------------------------------------------
def glr_forward(x, g, cuts, h0, gw):
    """h [rows, D], hT [P, D] and their bounds. A row adds 8 u of what it joins: 4 u + |g| u of the gate's exponential
    (the tests' gates lie within 2.6 of 0, or give exactly 0), one of the gates' product or of the fused
    multiply-add, and its share of the join of its span."""
    a = np.repeat(np.exp(g), gw, axis=1)
    h, e = np.zeros_like(x), np.zeros_like(x)
    hT, eT = h0.copy(), np.zeros_like(h0)
    for p in range(len(cuts) - 1):
        cur, mag, err = h0[p].copy(), np.abs(h0[p]), np.zeros_like(h0[p])
        for t in range(cuts[p], cuts[p + 1]):
            cur = a[t] * cur + x[t]
            mag = a[t] * mag + np.abs(x[t])
            err = a[t] * err + 8 * U * mag
            h[t], e[t] = cur, err
        hT[p], eT[p] = cur, err
    return h, e, hT, eT


def glr_backward(x, g, cuts, h0, gw, dy, dhT):
    """dx, dg, dh0 and their bounds (the same recurrence from the end; dg a product of two bounded numbers)."""
    a = np.repeat(np.exp(g), gw, axis=1)
    h, he, _, _ = glr_forward(x, g, cuts, h0, gw)
    dx, dxe, d, de = (np.zeros_like(x) for _ in range(4))
    dh0, dh0e = dhT.copy(), np.zeros_like(dhT)
    for p in range(len(cuts) - 1):
        m, mag, err = dhT[p].copy(), np.abs(dhT[p]), np.zeros_like(dhT[p])
        for t in range(cuts[p + 1] - 1, cuts[p] - 1, -1):
            lam, lmag = dy[t] + m, np.abs(dy[t]) + mag
            dx[t], dxe[t] = lam, err + U * lmag
            prev, preve = (h[t - 1], he[t - 1]) if t > cuts[p] else (h0[p], np.zeros_like(h0[p]))
            m, mag = a[t] * lam, a[t] * lmag
            err = a[t] * err + 8 * U * mag
            d[t] = m * prev
            de[t] = err * (np.abs(prev) + preve) + mag * preve + 2 * U * mag * np.abs(prev)
        dh0[p], dh0e[p] = m, err
    rows, H = g.shape
    dd, dde = d.reshape(rows, H, gw), de.reshape(rows, H, gw)
    return dx, dxe, dd.sum(2), dde.sum(2) + gw * U * (np.abs(dd) + dde).sum(2), dh0, dh0e


# ---- norm and rotation -------------------------------------------------------------------------------
def pairs(rd, layout):
    i = np.arange(rd // 2)
    return (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + rd // 2)


def turn(v, cos, sin, rd, layout, sign):
    """The rotation of v [T, H, hd] and the sum of the magnitudes of what it adds."""
    a, b = pairs(rd, layout)
    c, s = cos[:, None, :], sign * sin[:, None, :]
    o, m = v.copy(), np.abs(v)
    o[..., a], o[..., b] = v[..., a] * c - v[..., b] * s, v[..., b] * c + v[..., a] * s
    m[..., a] = np.abs(v[..., a] * c) + np.abs(v[..., b] * s)
    m[..., b] = np.abs(v[..., b] * c) + np.abs(v[..., a] * s)
    return o, m


def rope_head(x, w, pos, table, rd, layout, norm, eps, dout=None):
    """One kind's heads: out and its bound, and with dout also dx, dw and theirs. r carries hd / 2 u of the sum of
    squares, 4 u of rsqrtf and a few of its argument; each product one more."""
    T, H, hd = x.shape
    tab = table[np.clip(pos, 0, len(table) - 1)]
    cos, sin = tab[:, :rd // 2], tab[:, rd // 2:]
    pad = ((pos < 0) | (pos >= len(table)))[:, None, None]
    w = np.ones(hd) if w is None or not norm else w
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps) if norm else np.ones((T, H, 1))
    out, mag = turn(x * r * w, cos, sin, rd, layout, 1.0)
    res = [np.where(pad, 0.0, out), np.where(pad, 0.0, (hd / 2 + 16) * U * mag)]
    if dout is None:
        return res
    e, em = turn(dout, cos, sin, rd, layout, -1.0)
    rows = T * H
    dw = np.where(pad, 0.0, e * x * r).sum((0, 1))
    dwe = (rows + hd / 2 + 16) * U * np.where(pad, 0.0, em * np.abs(x) * r).sum((0, 1))
    t, tm = e * w, em * np.abs(w)
    k = (t * x).mean(-1, keepdims=True) if norm else 0.0
    km = (tm * np.abs(x)).mean(-1, keepdims=True) if norm else 0.0
    dx = r * (t - x * r * r * k)
    dxe = (2 * hd + 32) * U * r * (tm + np.abs(x) * r * r * km)
    return res + [np.where(pad, 0.0, dx), np.where(pad, 0.0, dxe), dw, dwe]


# ---- log probabilities -------------------------------------------------------------------------------
def logprobs(x, targets, scale):
    """logs [N, V], logp, entropy, lse and the bounds of the last three and of logs. A term 2^t has 4 u of exp2f and
    the error of its exponent, 3 u |t| (t within R / ln 2 of 0); the sum has V u in the worst order."""
    z = x * scale
    m = z.max(1, keepdims=True)
    empty = np.isneginf(m)
    with np.errstate(invalid="ignore", divide="ignore"):
        d = np.where(empty, -np.inf, z - m)
        s = np.exp(d).sum(1, keepdims=True)
        lse = np.where(empty, -np.inf, m + np.log(s))
        logs = np.where(empty, -np.inf, d - np.log(s))
        p = np.exp(logs)
        H = -np.where(p > 0, p * logs, 0.0).sum(1)
    V = x.shape[1]
    live = p > 1e-30
    R = np.where(live, np.abs(np.where(live, logs, 0.0)), 0.0).max(1)
    rel = (8 * R + V + 64) * U
    given = (targets >= 0) & (targets < V)
    pick = logs[np.arange(len(x)), np.where(given, targets, 0)]
    logp = np.where(given, pick, 0.0)
    fin = np.where(np.isfinite(logs), logs, 0.0)
    logs_e = rel[:, None] + 8 * U * np.abs(fin)
    lse_f = np.where(np.isfinite(lse[:, 0]), lse[:, 0], 0.0)
    return {"logs": logs, "logs_e": logs_e, "p": p, "logp": logp,
            "logp_e": rel + 8 * U * np.where(np.isfinite(logp), np.abs(logp), 0.0), "H": H, "H_e": rel * (2 + R + H),
            "lse": lse[:, 0], "lse_e": rel + 8 * U * np.abs(lse_f), "R": R}


def logprobs_backward(x, targets, scale, d_logp, d_entropy):
    """dlogits and its bound: p has the error of z - lse as the forward stored it, 8 u of |z| + |lse| and the lse's
    own; beyond 1024 the differences are taken from the largest logit, and the same bound holds with R."""
    f = logprobs(x, targets, scale)
    N, V = x.shape
    given = (targets >= 0) & (targets < V)
    dl = np.where(given, d_logp, 0.0)[:, None]
    dh = np.zeros((N, 1)) if d_entropy is None else d_entropy[:, None]
    one = np.zeros((N, V))
    one[np.arange(N)[given], targets[given]] = 1.0
    p = f["p"]
    live = p > 0
    logs = np.where(live, f["logs"], 0.0)
    H = f["H"][:, None]
    dz = dl * (one - p) - dh * np.where(live, p * (logs + H), 0.0)
    lse = np.where(np.abs(f["lse"]) < 1024, np.abs(f["lse"]), 0.0)
    d_e = f["lse_e"] * (np.abs(f["lse"]) < 1024) + (8 * (2 * lse + f["R"]) + V + 64) * U
    rel = d_e[:, None] + 8 * U * np.abs(logs) + 16 * U
    tol = p * rel * (np.abs(dl) + np.abs(dh) * (np.abs(logs) + H + 2)) + p * np.abs(dh) * f["H_e"][:, None]
    tol = tol + 4 * U * np.abs(dl) * one
    return scale * dz, abs(scale) * tol + 4 * U * np.abs(scale * dz)


def order_topk(x, K):
    """The ids of the K largest of every row, the lower id first among equals."""
    return np.stack([np.lexsort((np.arange(len(r)), -(r + 0.0)))[:K] for r in x])
