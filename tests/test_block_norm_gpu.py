"""The norms around a block (sdm_block_norm, sdm_block_norm_backward) against their definition in 64 bits, and the gradients also
against differences. Bounds follow the arithmetic (u = 2^-24): a sum of n terms in any order is within n u of the sum of their
magnitudes, a root of a mean of squares carries half of that, expf and divisions are within 4 u."""

import numpy as np
import pytest
import torch

import sparse_slot_memory_gb300 as sdm
from operators_testlib import U, check, f64

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5


def act_of(kind, z):
    t = np.exp(-np.abs(z))
    sg, rest = np.where(z >= 0, 1, t) / (1 + t), np.where(z >= 0, t, 1) / (1 + t)
    if kind == "sigmoid":
        return sg, sg * rest, sg * rest
    with np.errstate(invalid="ignore"):   # at an infinite gate their limits
        act, bend = np.where(sg == 0, 0.0, z * sg), np.where((sg == 0) | (rest == 0), 0.0, z * sg * rest)
    return act, sg + bend, sg + np.abs(bend)   # and the magnitude of what the slope adds


def oracle(c, r, s):
    """Values and bounds from the inputs and r as the forward stored it."""
    x = {k: f64(v) for k, v in c.items() if isinstance(v, torch.Tensor)}
    n, D = x["o"].shape
    G = s.group or D
    ones = np.ones(D)
    wp = np.tile(x["w_post"], D // G) if "w_post" in x else ones
    wn, cs = x.get("w_pre", ones), x.get("cs", ones)

    def mean(v, width):
        return np.repeat(v.reshape(n, D // width, width).mean(2), width, axis=1)

    p = 1 / np.sqrt(mean(x["o"] ** 2, G) + EPS) if s.post else np.ones((n, D))
    h = x["o"] * p
    m = h * wp if s.post else x["o"]
    act, slope, smag = act_of(s.gate, x["z"]) if s.gate != "none" else (np.ones((n, D)), np.zeros((n, D)), np.zeros((n, D)))
    nn = m * act
    R = x.get("x", 0.0) + s.scale * cs * nn
    rel = (G / 2 + 48) * U
    val, tol = {"r": R}, {"r": rel * np.abs(s.scale * cs * nn) + U * np.abs(R)}
    dR, dRe = x.get("dr", np.zeros((n, D))), 0.0
    if s.pre:
        q = 1 / np.sqrt((r ** 2).mean(1, keepdims=True) + EPS)
        val["y"], tol["y"] = r * q * wn, (D / 2 + 16) * U * np.abs(r * q * wn)
        if "dy" in x:
            u = x["dy"] * wn
            k, km = (u * r).mean(1, keepdims=True), np.abs(u * r).mean(1, keepdims=True)
            dRe = (2 * D + 32) * U * q * (np.abs(u) + np.abs(r) * q * q * km) + U * np.abs(dR)
            dR = dR + q * (u - r * q * q * k)
            e = np.abs(x["dy"] * r * q)
            val["dw_pre"], tol["dw_pre"] = (x["dy"] * r * q).sum(0), (n + D / 2 + 16) * U * e.sum(0)
    if "do" in c:
        dRe = dRe + 2 * U * np.abs(dR)
        val["dx"], tol["dx"] = dR, dRe + np.zeros((n, D))
        sc = np.abs(s.scale * cs)
        e = np.abs(s.scale * dR * nn)
        val["dcs"], tol["dcs"] = (s.scale * dR * nn).sum(0), (np.abs(s.scale * nn) * dRe + rel * e).sum(0) + n * U * e.sum(0)
        dn = s.scale * cs * dR
        val["dz"], tol["dz"] = dn * m * slope, sc * np.abs(m) * (np.abs(slope) * dRe + (rel + 16 * U) * smag * np.abs(dR))
        v = dn * act * (wp if s.post else 1.0)
        ve = np.abs(wp if s.post else 1.0) * np.abs(act) * sc * (dRe + 32 * U * np.abs(dR))
        if s.post:
            g = dn * act * h
            ge = np.abs(act * h) * sc * dRe + rel * np.abs(g) + n * U * np.abs(g)
            val["dw_post"], tol["dw_post"] = g.sum(0).reshape(-1, G).sum(0), (ge + D / G * U * np.abs(g)).sum(0).reshape(-1, G).sum(0)
            k, km, ke = mean(v * x["o"], G), mean(np.abs(v * x["o"]), G), mean(ve * np.abs(x["o"]), G)
            val["do"] = p * (v - x["o"] * p * p * k)
            tol["do"] = p * (ve + np.abs(x["o"]) * p * p * ke) + (2 * G + 64) * U * p * (np.abs(v) + np.abs(x["o"]) * p * p * km)
        else:
            val["do"], tol["do"] = v, ve
    return val, tol


def case(rows, D, group=0, post=True, gate="none", res=True, cs=True, pre=True, xt="bf16", pad=0, weights=True, dr=True, seed=0):
    gen = torch.Generator().manual_seed(seed)
    s = sdm.BlockNormSpec(rows=rows, D=D, group=group, post=post, gate=gate, residual=res, pre=pre, scale=0.75, dtype=xt, eps=EPS)

    def wide(scale=1.0):
        t = torch.full((rows, D + pad), float("nan"))
        t[:, :D] = torch.randn(rows, D, generator=gen) * scale
        return t.to(DT[xt]).cuda()[:, :D]

    c = {"o": wide(0.8)}
    if gate != "none":
        c["z"] = wide(2.0)
    if res:
        c["x"] = wide(2.0)
    if weights:
        if post:
            c["w_post"] = torch.randn(group or D, generator=gen).cuda()
        if pre:
            c["w_pre"] = torch.randn(D, generator=gen).cuda()
        if cs:
            c["cs"] = torch.randn(D, generator=gen).cuda()
    if dr or not pre:
        c["dr"] = wide()
    if pre:
        c["dy"] = wide()
    return s, c


def run(s, c, pad=0, train=True):
    def out(*shape, t=torch.float32):
        return torch.full(shape, float("nan"), dtype=t, device="cuda")

    def row():
        return out(s.rows, s.D + pad, t=DT[s.dtype])[:, :s.D]

    r = {"r": row()}
    if s.pre:
        r["y"] = row()
    sdm.block_norm(s, c["o"], r["r"], x=c.get("x"), z=c.get("z"), y=r.get("y"), w_post=c.get("w_post"), w_pre=c.get("w_pre"),
                   channel_scale=c.get("cs"))
    if train:
        c["do"] = None
        r |= {"do": row(), "dx": row(), "dcs": out(s.D)}
        if s.gate != "none":
            r["dz"] = row()
        if s.post:
            r["dw_post"] = out(s.group or s.D)
        if s.pre:
            r["dw_pre"] = out(s.D)
        ws = sdm.alloc_block_norm_workspace(s)
        ws.fill_(255)
        sdm.block_norm_backward(s, c["o"], r["r"], c.get("dr"), r["do"], ws, z=c.get("z"), dy=c.get("dy"), w_post=c.get("w_post"),
                                w_pre=c.get("w_pre"), channel_scale=c.get("cs"), dx=r["dx"], dz=r.get("dz"),
                                dw_post=r.get("dw_post"), dw_pre=r.get("dw_pre"), d_channel_scale=r["dcs"])
    return r


def compare(s, c, r):
    val, tol = oracle(c, f64(r["r"]), s)
    for n in r:
        check(n, r[n], val[n], tol[n], torch.float32 if n in ("dw_post", "dw_pre", "dcs") else DT[s.dtype])


CASES = {
    "one": dict(rows=1, D=4), "narrow": dict(rows=77, D=8, gate="silu"), "d36": dict(rows=9, D=36, xt="f32"), "d100": dict(rows=33, D=100),
    "d512": dict(rows=40, D=512, gate="sigmoid"), "d516": dict(rows=11, D=516, xt="f32", gate="silu"), "d1500": dict(rows=13, D=1500),
    "d2048": dict(rows=700, D=2048, gate="silu"), "d4096": dict(rows=5, D=4096, gate="sigmoid", xt="f32"), "d8192": dict(rows=3, D=8192, gate="silu"),
    "d8200": dict(rows=4, D=8200, gate="silu"), "d16384": dict(rows=3, D=16384, xt="f32", gate="sigmoid"),
    # groups: within a warp, of warps, of odd widths, several rows to a block
    "g4": dict(rows=50, D=64, group=4, xt="f32"), "g120": dict(rows=21, D=1920, group=120, gate="silu"), "g120_alone": dict(rows=21, D=1920, group=120, gate="silu", res=False, pre=False, cs=False),
    "g128": dict(rows=300, D=512, group=128, xt="f32"), "g256": dict(rows=9, D=2048, group=256), "g516": dict(rows=4, D=7740, group=516, gate="sigmoid"),
    "g1024": dict(rows=5, D=4096, group=1024, xt="f32"), "g36": dict(rows=90, D=252, group=36), "g712": dict(rows=6, D=4984, group=712),
    # parts left out
    "no_post": dict(rows=20, D=260, post=False), "no_pre": dict(rows=20, D=260, pre=False, gate="silu"), "no_res": dict(rows=20, D=260, res=False),
    "sum": dict(rows=20, D=260, post=False, cs=False), "bare": dict(rows=20, D=64, post=False, res=False, pre=False, weights=False),
    "no_weights": dict(rows=20, D=260, weights=False, gate="sigmoid"), "no_dr": dict(rows=20, D=260, dr=False, xt="f32"),
    "strided": dict(rows=20, D=132, pad=4, gate="silu"), "strided_f32": dict(rows=7, D=1000, pad=12, xt="f32"),
}


@pytest.mark.parametrize("name", list(CASES))
def test_forward_and_backward(name):
    s, c = case(**CASES[name])
    compare(s, c, run(s, c, CASES[name].get("pad", 0)))


def test_no_rows():
    s, c = case(0, 64)
    r = run(s, c)
    assert all(bool((r[n] == 0).all()) for n in ("dw_post", "dw_pre", "dcs"))


def test_gates_at_the_ends():
    """Gates of any size, infinite ones too, give 0, 1 or themselves, and no NaN."""
    for gate in ("sigmoid", "silu"):
        s, c = case(4, 64, gate=gate, xt="f32", pre=False)
        big = torch.tensor([float("-inf"), -3e38, -1000.0, -104.0, -90.0, 0.0, 90.0, 1000.0], device="cuda").repeat(8)
        c["z"][:] = big
        compare(s, c, run(s, c))
    s, c = case(2, 64, gate="sigmoid", xt="f32")
    c["z"][:] = float("inf")
    compare(s, c, run(s, c))


def test_rows_of_zeros_and_of_large_values():
    s, c = case(4, 260, xt="f32", gate="none")
    c["o"][0], c["x"][0] = 0.0, 0.0
    c["o"][1] *= 1e15
    c["x"][2] *= 1e15
    compare(s, c, run(s, c))


def test_nan_stays_in_its_row():
    s, c = case(40, 132, gate="silu")
    clean = run(s, c)
    c["o"][7, 3] = float("nan")
    c["x"][21, 5] = float("inf")
    r = run(s, c)
    rows = [i for i in range(40) if i not in (7, 21)]
    for n in ("r", "y", "do", "dz", "dx"):
        assert torch.equal(r[n][rows], clean[n][rows]), n
    assert bool(r["r"][7].isnan().all()) and bool(r["y"][21].isnan().any())


def test_in_place():
    """The stream, the block's output and the gradients may be written where they were read."""
    s, c = case(50, 516, gate="silu")
    want = run(s, c)
    x, o = c["x"].clone(), c["o"].clone()
    sdm.block_norm(s, o, x, x=x, z=c["z"], y=o, w_post=c["w_post"], w_pre=c["w_pre"], channel_scale=c["cs"])
    assert torch.equal(x, want["r"]) and torch.equal(o, want["y"])
    dr, z, o = c["dr"].clone(), c["z"].clone(), c["o"].clone()
    sdm.block_norm_backward(s, o, want["r"], dr, o, z=z, dy=c["dy"], w_post=c["w_post"], w_pre=c["w_pre"], channel_scale=c["cs"], dx=dr,
                            dz=z)
    assert torch.equal(dr, want["dx"]) and torch.equal(z, want["dz"]) and torch.equal(o, want["do"])


def test_in_place_wide_rows():
    s, c = case(3, 12000, gate="sigmoid", xt="f32")
    want = run(s, c)
    dr, z, o = c["dr"].clone(), c["z"].clone(), c["o"].clone()
    sdm.block_norm_backward(s, o, want["r"], dr, o, z=z, dy=c["dy"], w_post=c["w_post"], w_pre=c["w_pre"], channel_scale=c["cs"], dx=dr,
                            dz=z)
    assert torch.equal(dr, want["dx"]) and torch.equal(z, want["dz"]) and torch.equal(o, want["do"])


def test_runs_are_bitwise_equal_and_rows_independent():
    s, c = case(3000, 260, gate="silu")
    a, b = run(s, c), run(s, c)
    assert all(torch.equal(a[n], b[n]) for n in a)
    part, _ = case(7, 260, gate="silu")
    r = run(part, {k: (v[100:107] if v is not None and v.dim() == 2 else v) for k, v in c.items()})
    assert all(torch.equal(r[n], a[n][100:107]) for n in ("r", "y", "do", "dz", "dx"))


def test_gradients_against_differences():
    """Central differences of the definition in 64 bits against the kernel's gradients (float32 rows, so r is nearly not rounded:
    u of its magnitude, which the step of 1e-4 sees as 1e-3 of u / 1e-4)."""
    s, c = case(3, 32, group=8, gate="silu", xt="f32")
    r = run(s, c)
    x = {k: f64(v) for k, v in c.items() if v is not None}

    def loss(v):
        n, D, G = 3, 32, 8
        h = v["o"].reshape(n, D // G, G)
        m = (h / np.sqrt((h ** 2).mean(2, keepdims=True) + EPS) * v["w_post"]).reshape(n, D)
        R = v["x"] + 0.75 * v["cs"] * m * v["z"] / (1 + np.exp(-v["z"]))
        y = R / np.sqrt((R ** 2).mean(1, keepdims=True) + EPS) * v["w_pre"]
        return (R * x["dr"]).sum() + (y * x["dy"]).sum()

    rng = np.random.default_rng(1)
    for n, d in (("o", "do"), ("z", "dz"), ("x", "dx"), ("w_post", "dw_post"), ("w_pre", "dw_pre"), ("cs", "dcs")):
        u = rng.standard_normal(x[n].shape)
        e = 1e-4
        diff = (loss(x | {n: x[n] + e * u}) - loss(x | {n: x[n] - e * u})) / (2 * e)
        got = (f64(r[d]) * u).sum()
        # the third derivative over 6, e^2 of it; the kernel's own error
        assert abs(diff - got) <= 1e-5 * (np.abs(f64(r[d]) * u).sum() + 10), (n, diff, got)


def test_more_than_2_31_elements():
    rows, D = 140000, 16384
    s = sdm.BlockNormSpec(rows=rows, D=D, post=False, residual=True, pre=True)
    o = torch.empty(rows, D, dtype=torch.bfloat16, device="cuda").normal_()
    y, r = torch.empty_like(o), torch.empty_like(o)
    sdm.block_norm(s, o, r, x=o, y=y)
    part = sdm.BlockNormSpec(rows=5, D=D, post=False, residual=True, pre=True)
    ry, rr = torch.empty_like(o[-5:]), torch.empty_like(o[-5:])
    sdm.block_norm(part, o[-5:], rr, x=o[-5:], y=ry)
    assert torch.equal(rr, r[-5:]) and torch.equal(ry, y[-5:]) and not bool(ry.isnan().any())
