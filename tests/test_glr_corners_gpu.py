"""Corners of the gated linear recurrence: rows that belong to no sequence, outputs in place of inputs, and gates of -inf, NaN and
infinities in sequences that several blocks walk."""

import numpy as np
import pytest
import torch

import sparse_slot_memory_gb300 as sdm
from operators_testlib import check, f64, glr_backward, glr_forward
from operators_testlib import check as bound

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def case(rows, cuts, D, gw, xt="f32", gt="f32", seed=0, mean=3.0):
    """Sequences between the `cuts` of `rows` rows, their states and their gradients."""
    gen = torch.Generator().manual_seed(seed)
    P, H = len(cuts) - 1, D // gw
    c = {"spec": sdm.GlrSpec(P=P, rows=rows, D=D, gate_width=gw, x_dtype=xt, g_dtype=gt), "gw": gw,
         "cuts": np.asarray(cuts, np.int64)}
    c["x"], c["dy"] = (torch.randn(rows, D, generator=gen).to(DT[xt]).cuda() for _ in range(2))
    c["g"] = torch.nn.functional.logsigmoid(torch.randn(rows, H, generator=gen) + mean).to(DT[gt]).cuda()
    c["offsets"] = torch.from_numpy(c["cuts"]).cuda()
    c["h0"], c["dhT"] = (torch.randn(P, D, generator=gen).cuda() for _ in range(2))
    return c


def run(c, fill=float("nan")):
    """Every output full of `fill` beforehand, and so the states and the workspace."""
    s = c["spec"]
    r = {k: torch.full_like(c["x"], fill) for k in ("y", "dx")}
    r["dg"] = torch.full_like(c["g"], fill)
    r["hT"], r["dh0"] = (torch.full_like(c["h0"], fill) for _ in range(2))
    states, ws = sdm.alloc_glr_states(s).fill_(fill), sdm.alloc_glr_workspace(s)
    ws[:ws.numel() // 4 * 4].view(torch.float32).fill_(fill)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sdm.glr_forward(s, c["x"], c["g"], r["y"], offsets=c["offsets"], h0=c["h0"], hT=r["hT"], states=states, status=st)
    sdm.glr_backward(s, c["x"], c["g"], c["dy"], states, r["dx"], r["dg"], ws, offsets=c["offsets"], dhT=c["dhT"],
                     dh0=r["dh0"], status=st)
    r["status"] = int(st.item())
    return r


def finite(v):
    """v with NaN in the place of infinities."""
    if isinstance(v, torch.Tensor):
        return torch.where(torch.isfinite(v), v, float("nan"))
    return np.where(np.isfinite(v), v, np.nan)


def compare(c, r, rows=slice(None), kinds=True):
    """`kinds`: infinities and NaN are told apart."""
    s, cuts = c["spec"], c["cuts"]
    check = lambda name, got, want, *tol: bound(name, *((got, want) if kinds else (finite(got), finite(want))), *tol)
    x, g, dy, h0, dhT = (f64(c[k]) for k in ("x", "g", "dy", "h0", "dhT"))
    with np.errstate(invalid="ignore"):
        h, he, hT, hTe = glr_forward(x, g, cuts, h0, c["gw"])
        dx, dxe, dg, dge, dh0, dh0e = glr_backward(x, g, cuts, h0, c["gw"], dy, dhT)
        check("y", r["y"][rows], h[rows], he[rows], DT[s.x_dtype])
        check("hT", r["hT"], hT, hTe)
        check("dx", r["dx"][rows], dx[rows], dxe[rows], DT[s.x_dtype])
        check("dg", r["dg"][rows], dg[rows], dge[rows], DT[s.g_dtype])
        check("dh0", r["dh0"], dh0, dh0e)


@pytest.mark.parametrize("D, gw", [(264, 1), (256, 64), (512, 256), (264, 132)])
@pytest.mark.parametrize("rows, cuts", [(500, [70, 70, 300, 431]), (9000, [100, 8500]), (40, [0, 10, 30]), (30, [12, 12])])
def test_rows_of_no_sequence_stay_as_they_are(rows, cuts, D, gw):
    """Offsets may leave rows before the first and behind the last sequence (a packed batch's padding), whatever the
    heads' width is: nothing is written there, and nothing read."""
    c = case(rows, cuts, D, gw)
    inside = slice(cuts[0], cuts[-1])
    outside = torch.ones(rows, dtype=torch.bool, device="cuda")
    outside[inside] = False
    for k in ("x", "g", "dy"):
        c[k][outside] = float("nan")
    for fill in (float("nan"), 7.0):
        r = run(c, fill)
        assert r["status"] == 0
        for k in ("y", "dx", "dg"):
            assert bool((torch.isnan(r[k][outside]) if fill != fill else r[k][outside] == fill).all()), k
        compare(c, r, inside)


@pytest.mark.parametrize("xt, gt", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows, cuts, D, gw", [(9001, [0, 9001], 12, 4), (8400, [0, 4200, 8400], 132, 1), (300, [0, 300], 132, 1),
                                               (12000, [0, 0, 9000, 9003, 12000], 64, 1)])
def test_outputs_in_place_of_inputs(rows, cuts, D, gw, xt, gt):
    """y over x, dx over dy and dx over x, also where rows of other places are divided into segments."""
    c = case(rows, cuts, D, gw, xt, gt, seed=2)
    s, want = c["spec"], run(c)
    compare(c, want)
    X, G, H0 = f64(c["x"]), f64(c["g"]), f64(c["h0"])
    y, states, hT = c["x"].clone(), sdm.alloc_glr_states(s), torch.empty_like(c["h0"])
    sdm.glr_forward(s, y, c["g"], y, offsets=c["offsets"], h0=c["h0"], hT=hT, states=states)
    h, he, last, laste = glr_forward(X, G, c["cuts"], H0, gw)
    check("y", y, h, he, DT[xt])
    check("hT", hT, last, laste)
    dx, dxe, dg, dge, dh0, dh0e = glr_backward(X, G, c["cuts"], H0, gw, f64(c["dy"]), f64(c["dhT"]))
    for over in ("dy", "x"):
        args = {k: c[k].clone() for k in ("x", "dy")}
        out, got, first = args[over], torch.empty_like(c["g"]), torch.empty_like(c["h0"])
        sdm.glr_backward(s, args["x"], c["g"], args["dy"], states, out, got, offsets=c["offsets"], dhT=c["dhT"], dh0=first)
        check("dx", out, dx, dxe, DT[xt])
        check("dg", got, dg, dge, DT[gt])
        check("dh0", first, dh0, dh0e)


@pytest.mark.parametrize("xt, gt", [("f32", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows, cuts, D, gw", [
    (9001, [0, 9001], 12, 1), (9001, [0, 9001], 24, 12), (20000, [0, 9000, 9003, 20000], 64, 1),   # segments
    (2100, [0, 700, 1400, 2100], 2048, 1), (700, [0, 300, 700], 2048, 128)])                        # clusters
@pytest.mark.parametrize("mean, values", [(3.0, "nan"), (3.0, "inf"), (9.0, "inf")])
def test_resets_nan_and_infinity_over_divided_sequences(rows, cuts, D, gw, xt, gt, mean, values):
    """Gates of -inf and of 0, NaN or infinite inputs and gradients, in sequences that several blocks walk: they reach what
    the definition says and nothing else. Infinities stay infinities while the gates' products stay in range (mean 9:
    about e^-4 over all rows); past it they may be NaN."""
    c = case(rows, cuts, D, gw, xt, gt, seed=5, mean=mean)
    gen = torch.Generator().manual_seed(6)
    for t in torch.randint(0, rows, (6,), generator=gen).tolist() + [cuts[1] - 1, cuts[1] % rows, 0, 64, 255, 256]:
        c["g"][t, torch.randint(0, D // gw, (1,), generator=gen).item()] = -float("inf")
    c["g"][rows // 2] = -float("inf")       # every channel of a row
    c["g"][rows // 3:rows // 3 + 70] = 0.0
    for value in (float("nan"),) if values == "nan" else (float("inf"), -float("inf")):
        t, ch = torch.randint(0, rows, (2,), generator=gen).tolist(), torch.randint(0, D, (2,), generator=gen).tolist()
        c["x"][t[0], ch[0]], c["dy"][t[1], ch[1]] = value, value
    compare(c, run(c), kinds=mean > 3.0 or values == "nan")
