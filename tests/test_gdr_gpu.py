"""The gated delta rule (sdm_gdr_forward, sdm_gdr_backward, sdm_gdr_step) against its definition in 64 bits
(tests/gdr_testlib.py, which derives the bounds), and the gradients also against differences."""

import numpy as np
import pytest
import torch

import sparse_slot_memory_gb300 as sdm
from gdr_testlib import backward, forward, oracle
from operators_testlib import U, check, f64
from sparse_slot_memory_gb300 import _abi

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def case(lens, Hk=1, Hv=1, dk=64, dv=64, xt="bf16", gt="f32", pad=0, state=True, rate=0.3, seed=0, before=0, behind=0, alike=0.3):
    """Queries and keys of length 1 at most (keys that have `alike` in common), slices of rows `pad` heads wider."""
    gen = torch.Generator().manual_seed(seed)
    n, P = sum(lens) + before + behind, len(lens)

    def heads(H, d, length=None):
        t = torch.randn(n, H, d, generator=gen)
        if length is not None:
            t = t + length * torch.randn(1, H, d, generator=gen)
            t = t / t.norm(dim=2, keepdim=True) * (1 - 2.0 ** -7)
        wide = torch.full((n, H + pad, d), float("nan"))
        wide[:, :H] = t
        return wide.to(DT[xt]).cuda()[:, :H]

    c = {"spec": sdm.GdrSpec(P=P, rows=n, k_heads=Hk, v_heads=Hv, dk=dk, dv=dv, x_dtype=xt, g_dtype=gt, scale=dk ** -0.5)}
    c["q"], c["k"], c["v"], c["dy"] = heads(Hk, dk, 0.0), heads(Hk, dk, alike), heads(Hv, dv), heads(Hv, dv)
    for name, value in (("g", -rate * torch.nn.functional.softplus(torch.randn(n, Hv, generator=gen))),
                        ("beta", torch.sigmoid(torch.randn(n, Hv, generator=gen)))):
        c[name] = torch.full((n, Hv + pad), float("nan"), dtype=DT[gt], device="cuda")[:, :Hv]
        c[name].copy_(value)
    c["cuts"] = before + np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    c["offsets"] = None if len(set(lens)) == 1 and not before + behind else torch.from_numpy(c["cuts"]).cuda()
    for name in ("h0", "dhT"):
        c[name] = torch.randn(P, Hv, dk, dv, generator=gen).cuda() * 0.5 if state else None
    c["pad"] = pad
    return c


def outputs(c, train=True):
    s, pad = c["spec"], c["pad"]

    def nan(*shape, t=torch.float32):
        return torch.full(shape, float("nan"), dtype=t, device="cuda")

    xt, gt = DT[s.x_dtype], DT[s.g_dtype]
    r = {"y": nan(s.rows, s.v_heads + pad, s.dv, t=xt)[:, :s.v_heads], "hT": nan(s.P, s.v_heads, s.dk, s.dv)}
    if train:
        r |= {"dq": nan(s.rows, s.k_heads + pad, s.dk, t=xt)[:, :s.k_heads], "dk": nan(s.rows, s.k_heads + pad, s.dk, t=xt)[:, :s.k_heads],
              "dv": nan(s.rows, s.v_heads + pad, s.dv, t=xt)[:, :s.v_heads], "dg": nan(s.rows, s.v_heads + pad, t=gt)[:, :s.v_heads],
              "dbeta": nan(s.rows, s.v_heads + pad, t=gt)[:, :s.v_heads], "dh0": nan(s.P, s.v_heads, s.dk, s.dv)}
    return r


def run(c, train=True):
    s, r = c["spec"], outputs(c, train)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = [c[n] for n in ("q", "k", "v", "g", "beta")]
    states = sdm.alloc_gdr_states(s) if train else None
    ws = sdm.alloc_gdr_workspace(s, backward=False)
    for t in (states, ws):
        if t is not None:
            t.fill_(255)
    sdm.gdr_forward(s, *x, r["y"], ws, offsets=c["offsets"], h0=c["h0"], hT=r["hT"], states=states, status=st)
    if train:
        ws = sdm.alloc_gdr_workspace(s)
        ws.fill_(255)
        sdm.gdr_backward(s, *x, c["dy"], states, *[r[n] for n in ("dq", "dk", "dv", "dg", "dbeta")], ws, offsets=c["offsets"],
                         dhT=c["dhT"], dh0=r["dh0"], status=st)
    assert int(st.item()) == 0
    return r


def compare(c, r, train=True, whole=True):
    s = c["spec"]
    x = {n: f64(c[n]) for n in ("q", "k", "v", "g", "beta", "dy")}
    for n in ("h0", "dhT"):
        x[n] = f64(c[n]) if c[n] is not None else np.zeros((s.P, s.v_heads, s.dk, s.dv))
    val, tol = oracle(x, c["cuts"], s.scale, s.x_dtype, train, whole)
    types = {"y": s.x_dtype, "dq": s.x_dtype, "dk": s.x_dtype, "dv": s.x_dtype, "dg": s.g_dtype, "dbeta": s.g_dtype}
    for n in r:
        check(n, r[n], val[n], tol[n], DT[types.get(n, "f32")])


CASES = {
    # one row, one less and more than a block, several blocks
    "t1": dict(lens=[1]), "t2": dict(lens=[2, 2], dk=8, dv=8), "t63": dict(lens=[63], dk=16, dv=24), "t64": dict(lens=[64, 64]),
    "t65": dict(lens=[65], dk=128, dv=128), "t200": dict(lens=[200], dk=128, dv=128, gt="bf16"),
    # head sizes on both sides of the tiles', value heads that share keys
    "d8": dict(lens=[70], dk=8, dv=128), "d128_8": dict(lens=[70], dk=128, dv=8), "d72_56": dict(lens=[130], Hk=2, Hv=6, dk=72, dv=56),
    "d120": dict(lens=[129], Hk=2, Hv=4, dk=120, dv=120, gt="bf16"), "d64_40": dict(lens=[100], Hk=3, Hv=3, dk=56, dv=40),
    "d96_112": dict(lens=[90], dk=96, dv=112, Hv=2),
    # float32 rows
    "f1": dict(lens=[1], xt="f32"), "f65": dict(lens=[65], xt="f32", dk=128, dv=128), "f130": dict(lens=[130], xt="f32", Hk=2, Hv=4, dk=72, dv=56),
    "f_ragged": dict(lens=[3, 0, 100, 64], xt="f32", dk=24, dv=40, gt="bf16", Hv=3),
    # ragged, with empty sequences first, last and between; rows of no sequence before and behind
    "ragged": dict(lens=[0, 5, 130, 0, 64, 1, 0], Hv=2), "outside": dict(lens=[70, 3], before=5, behind=9, Hk=2, Hv=4, dk=32, dv=32),
    "many": dict(lens=[1, 2, 0, 65] * 12, dk=16, dv=16), "empty": dict(lens=[0, 0]),
    # rows further apart than they are long; no states given; strong and no decay
    "strided": dict(lens=[100], Hk=2, Hv=4, pad=1), "strided_f32": dict(lens=[80], xt="f32", Hk=1, Hv=2, dk=32, dv=32, pad=2),
    "no_state": dict(lens=[90, 0, 2], state=False), "strong": dict(lens=[150], rate=12.0, xt="f32"), "strong_bf16": dict(lens=[150], rate=12.0),
    "keeps": dict(lens=[300], rate=0.0, dk=32, dv=32, xt="f32"),
}


@pytest.mark.parametrize("name", list(CASES))
def test_forward_and_backward(name):
    c = case(**CASES[name])
    compare(c, run(c))


@pytest.mark.parametrize("xt", ["bf16", "f32"])
def test_forward_alone(xt):
    c = case([130, 0, 7], Hk=1, Hv=2, dk=64, dv=48, xt=xt)
    compare(c, run(c, False), False)


@pytest.mark.parametrize("xt", ["bf16", "f32"])
def test_gates_of_minus_infinity_start_anew(xt):
    c = case([150, 40], Hv=2, dk=32, dv=32, xt=xt)
    c["g"][64, :] = -float("inf")
    c["g"][70:80, 0] = -float("inf")
    c["g"][90, 1] = torch.finfo(torch.float32).min
    c["g"][150, :] = -float("inf")   # a sequence's first row: its given state drops out
    r = run(c)
    compare(c, r)
    assert bool((r["dg"][64] == 0).all()) and bool((r["dg"][70:80, 0] == 0).all()) and bool((r["dh0"][1] == 0).all())


@pytest.mark.parametrize("xt", ["bf16", "f32"])
def test_write_strengths_of_zero_and_one(xt):
    """Rows of strength 0 write nothing and have a gradient of it; strengths of 1 overwrite what a key holds."""
    c = case([140], Hv=2, dk=32, dv=32, xt=xt)
    c["beta"][:, 0] = (torch.arange(140, device="cuda") % 3 != 0).float()
    c["beta"][30:70, 1] = 0.0
    compare(c, run(c))


def test_keys_that_are_all_the_same():
    """The triangular system at its worst: every row corrects what the row before has written."""
    for xt in ("bf16", "f32"):
        c = case([130], dk=32, dv=32, xt=xt, rate=0.0)
        k = torch.zeros(32)
        k[3] = 1.0
        c["k"].copy_(k.to(c["k"].dtype))
        c["beta"].fill_(1.0)
        compare(c, run(c))


def test_state_in_place_and_cut_sequences():
    """hT may be h0; a sequence cut in two calls agrees with one call within the bounds of both."""
    c = case([200], Hk=1, Hv=2, dk=64, dv=64)
    whole = run(c, False)
    s, state = c["spec"], c["h0"].clone()
    y = torch.empty_like(whole["y"])
    for a, b in ((0, 77), (77, 200)):
        part = sdm.GdrSpec(P=1, rows=b - a, k_heads=1, v_heads=2, dk=64, dv=64, scale=s.scale)
        sdm.gdr_forward(part, *[c[n][a:b] for n in ("q", "k", "v", "g", "beta")], y[a:b], sdm.alloc_gdr_workspace(part, backward=False),
                        h0=state, hT=state)
    compare(c, {"y": y, "hT": state}, False)


def test_dh0_in_place_of_dhT():
    c = case([100], dk=32, dv=32, xt="f32")
    s, r = c["spec"], outputs(c)
    states, ws = sdm.alloc_gdr_states(s), sdm.alloc_gdr_workspace(s)
    x = [c[n] for n in ("q", "k", "v", "g", "beta")]
    sdm.gdr_forward(s, *x, r["y"], ws, h0=c["h0"], hT=r["hT"], states=states)
    r["dh0"].copy_(c["dhT"])
    sdm.gdr_backward(s, *x, c["dy"], states, *[r[n] for n in ("dq", "dk", "dv", "dg", "dbeta")], ws, dhT=r["dh0"], dh0=r["dh0"])
    compare(c, r)


def test_runs_are_bitwise_equal():
    c = case([300, 0, 129], Hk=2, Hv=4, dk=72, dv=56)
    a, b = run(c), run(c)
    for n in a:
        assert torch.equal(a[n].nan_to_num(7.0), b[n].nan_to_num(7.0)), n


def test_rows_outside_stay():
    c = case([70, 3], before=5, behind=9, Hk=2, Hv=4, dk=32, dv=32)
    r = run(c)
    for n in ("y", "dq", "dk", "dv", "dg", "dbeta"):
        assert bool(r[n][:5].isnan().all()) and bool(r[n][-9:].isnan().all()), n


def test_bad_offsets_are_cut_and_reported():
    c = case([70, 30], dk=32, dv=32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = outputs(c, False)
    off = torch.tensor([-3, 70, 500], device="cuda")
    sdm.gdr_forward(c["spec"], *[c[n] for n in ("q", "k", "v", "g", "beta")], r["y"], sdm.alloc_gdr_workspace(c["spec"], backward=False),
                    offsets=off, h0=c["h0"], hT=r["hT"], status=st)
    assert int(st.item()) == _abi.SDM_DEV_BAD_OFFSET
    compare(c, r, False)


def test_gradients_against_differences():
    """Central differences of the 64-bit rule, along random directions, against the kernel's gradients: the step's error is below
    1e-6 of the sum's magnitude, the kernel's within its bounds."""
    c = case([70], Hk=1, Hv=2, dk=16, dv=16, xt="f32")
    r, s = run(c), c["spec"]
    x = {n: f64(c[n]) for n in ("q", "k", "v", "g", "beta", "h0")}
    dy, dhT = f64(c["dy"]), f64(c["dhT"])
    full = {n: f64(c[n]) for n in ("q", "k", "v", "g", "beta", "dy", "h0", "dhT")}
    _, tol = oracle(full, c["cuts"], s.scale, "f32")

    def loss(z):
        total = 0.0
        for h in range(2):
            y, states, _ = forward(z["q"][:, 0], z["k"][:, 0], z["v"][:, h], z["g"][:, h], z["beta"][:, h], z["h0"][0, h], s.scale)
            total += (y * dy[:, h]).sum() + (states[-1] * dhT[0, h]).sum()
        return total

    rng = np.random.default_rng(3)
    for n, d in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("beta", "dbeta"), ("h0", "dh0")):
        for _ in range(3):
            u = rng.standard_normal(x[n].shape)
            e = 1e-5
            diff = (loss(x | {n: x[n] + e * u}) - loss(x | {n: x[n] - e * u})) / (2 * e)
            got = (f64(r[d]) * u).sum()
            # third differences of the loss over 6, and the loss's own digits over the step
            lim = (tol[d] * abs(u)).sum() + 1e-6 * (abs(f64(r[d]) * u)).sum() + 1e-4
            assert abs(diff - got) <= lim, (n, diff, got, lim)


# ---- one token of every request ---------------------------------------------------------------------------------
STEP = {
    "plain": dict(B=3, Hk=1, Hv=2, dk=64, dv=64), "wide": dict(B=5, Hk=2, Hv=4, dk=128, dv=128), "odd": dict(B=4, Hk=2, Hv=6, dk=72, dv=56, xt="f32"),
    "narrow": dict(B=2, Hk=1, Hv=1, dk=8, dv=8), "tall": dict(B=2, Hk=1, Hv=1, dk=128, dv=8, gt="bf16"), "flat": dict(B=2, Hk=1, Hv=3, dk=8, dv=128, xt="f32"),
    "d120": dict(B=33, Hk=1, Hv=2, dk=120, dv=72, gt="bf16"), "one": dict(B=1, Hk=1, Hv=1, dk=64, dv=96),
}


@pytest.mark.parametrize("slots", [False, True])
@pytest.mark.parametrize("name", list(STEP))
def test_step(name, slots):
    kw = dict(STEP[name])
    B = kw.pop("B")
    c = case([1] * B, **kw, pad=1)
    s = c["spec"]
    gen = torch.Generator().manual_seed(5)
    n = B + 3
    state = torch.full((n, s.v_heads + 1, s.dk, s.dv), float("nan"), device="cuda")[:, :s.v_heads]   # rows further apart
    state.copy_(torch.randn(n, s.v_heads, s.dk, s.dv, generator=gen))
    start = state.clone()
    at = torch.randperm(n, generator=gen)[:B] if slots else torch.arange(B)
    if slots and B > 2:
        at[1] = -4
    y = outputs(c, False)["y"]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sdm.gdr_step(s, *[c[m] for m in ("q", "k", "v", "g", "beta")], state, y, slots=at.int().cuda() if slots else None, status=st)
    assert int(st.item()) == 0
    x = {m: f64(c[m]) for m in ("q", "k", "v", "g", "beta")}
    want, tol = f64(start).copy(), np.zeros(start.shape)
    wy, ty = np.zeros((B, s.v_heads, s.dv)), np.zeros((B, s.v_heads, s.dv))
    R = s.v_heads // s.k_heads
    for i in range(B):
        if at[i] < 0:
            continue
        for h in range(s.v_heads):
            q, k, v, g, b = x["q"][i, h // R], x["k"][i, h // R], x["v"][i, h], x["g"][i, h], x["beta"][i, h]
            S0 = f64(start[at[i], h])
            _, states, E = forward(q[None], k[None], v[None], np.array([g]), np.array([b]), S0, s.scale)
            want[at[i], h] = states[-1]
            wy[i, h] = s.scale * states[-1].T @ q
            # sums of dk terms in any order, exp within 4 u, a few products
            e = (s.dk + 16) * U
            mag = abs(v) + np.exp(g) * (abs(S0).T @ abs(k))
            tol[at[i], h] = e * (np.exp(g) * abs(S0) + 2 * np.outer(abs(k), b * mag))
            ty[i, h] = 2 * e * s.scale * (np.exp(g) * (abs(S0).T @ abs(q)) + (abs(k) @ abs(q)) * 2 * b * mag)
    check("y", y, wy, ty, DT[s.x_dtype])
    check("state", state, want, tol)


def test_step_refuses_slots_behind_the_table_and_leaves_padding_alone():
    c = case([1] * 4, dk=32, dv=32)
    s, state = c["spec"], torch.randn(3, 1, 32, 32, device="cuda")
    start, y = state.clone(), outputs(c, False)["y"]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sdm.gdr_step(s, *[c[m] for m in ("q", "k", "v", "g", "beta")], state, y, slots=torch.tensor([0, 3, -1, 2 ** 31 - 1], dtype=torch.int32).cuda(),
                 status=st)
    assert int(st.item()) == _abi.SDM_DEV_BAD_SLOT
    assert bool((y[1:] == 0).all()) and torch.equal(state[1:], start[1:]) and not torch.equal(state[0], start[0])


def test_steps_follow_a_prompt():
    """A prompt through the blocks, then tokens one at a time, against the rule over all of them."""
    c = case([100], Hk=2, Hv=4, dk=64, dv=64)
    s, n = c["spec"], 90
    y, state = torch.empty(100, 4, 64, dtype=torch.bfloat16, device="cuda"), c["h0"].clone()
    x = [c[m] for m in ("q", "k", "v", "g", "beta")]
    part = sdm.GdrSpec(P=1, rows=n, k_heads=2, v_heads=4, dk=64, dv=64, scale=s.scale)
    sdm.gdr_forward(part, *[t[:n] for t in x], y[:n], sdm.alloc_gdr_workspace(part, backward=False), h0=state, hT=state)
    one = sdm.GdrSpec(P=1, rows=1, k_heads=2, v_heads=4, dk=64, dv=64, scale=s.scale)
    for i in range(n, 100):
        sdm.gdr_step(one, *[t[i:i + 1] for t in x], state, y[i:i + 1])
    compare(c, {"y": y, "hT": state}, False)
