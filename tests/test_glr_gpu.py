"""The gated linear recurrence (sdm_glr_forward, sdm_glr_backward, sdm_glr_step) against its definition in 64 bits
(tests/operators_testlib.py, which derives the bounds), and the gradients also against differences."""

import numpy as np
import pytest
import torch

import sparse_slot_memory_gb300 as sdm
from operators_testlib import check, f64, glr_backward, glr_forward
from sparse_slot_memory_gb300 import _abi

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def rows(gen, n, cols, dtype, pad=0, scale=1.0):
    """A row array whose rows lie `pad` elements further apart than they are long."""
    t = torch.full((n, cols + pad), float("nan"), dtype=torch.float32)
    t[:, :cols] = torch.randn(n, cols, generator=gen) * scale
    return t.to(DT[dtype]).cuda()[:, :cols]


def case(lens, D, gw, xt="bf16", gt="f32", pad=0, state=True, mean=3.0, seed=0):
    gen = torch.Generator().manual_seed(seed)
    n, P, H = sum(lens), len(lens), D // gw
    c = {"spec": sdm.GlrSpec(P=P, rows=n, D=D, gate_width=gw, x_dtype=xt, g_dtype=gt), "gw": gw}
    c["x"], c["dy"] = rows(gen, n, D, xt, pad), rows(gen, n, D, xt, pad)
    z = torch.nn.functional.logsigmoid(torch.randn(n, H, generator=gen) + mean)
    c["g"] = torch.zeros(n, H + pad, dtype=DT[gt], device="cuda")[:, :H]
    c["g"].copy_(z)
    c["cuts"] = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    same = len(set(lens)) == 1
    c["offsets"] = None if same else torch.from_numpy(c["cuts"]).cuda()
    c["h0"] = torch.randn(P, D, generator=gen).cuda() if state else None
    c["dhT"] = torch.randn(P, D, generator=gen).cuda() if state else None
    return c


def out(n, cols, dtype, pad):
    return torch.full((n, cols + pad), float("nan"), dtype=DT[dtype], device="cuda")[:, :cols]


def run(c, pad=0):
    s = c["spec"]
    r = {"y": out(s.rows, s.D, s.x_dtype, pad), "hT": torch.full((s.P, s.D), float("nan"), device="cuda"),
         "dx": out(s.rows, s.D, s.x_dtype, pad), "dg": out(s.rows, s.gates, s.g_dtype, pad),
         "dh0": torch.full((s.P, s.D), float("nan"), device="cuda")}
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    states = sdm.alloc_glr_states(s)
    states.fill_(float("nan"))
    sdm.glr_forward(s, c["x"], c["g"], r["y"], offsets=c["offsets"], h0=c["h0"], hT=r["hT"], states=states, status=st)
    sdm.glr_backward(s, c["x"], c["g"], c["dy"], states, r["dx"], r["dg"], sdm.alloc_glr_workspace(s),
                     offsets=c["offsets"], dhT=c["dhT"], dh0=r["dh0"], status=st)
    assert int(st.item()) == 0
    return r


def compare(c, r):
    s = c["spec"]
    zero = np.zeros((s.P, s.D))
    h0 = f64(c["h0"]) if c["h0"] is not None else zero
    dhT = f64(c["dhT"]) if c["dhT"] is not None else zero
    x, g, dy = f64(c["x"]), f64(c["g"]), f64(c["dy"])
    h, he, hT, hTe = glr_forward(x, g, c["cuts"], h0, c["gw"])
    check("y", r["y"], h, he, DT[s.x_dtype])
    check("hT", r["hT"], hT, hTe)
    dx, dxe, dg, dge, dh0, dh0e = glr_backward(x, g, c["cuts"], h0, c["gw"], dy, dhT)
    check("dx", r["dx"], dx, dxe, DT[s.x_dtype])
    check("dg", r["dg"], dg, dge, DT[s.g_dtype])
    check("dh0", r["dh0"], dh0, dh0e)


CASES = {
    # one token, one row less and more than a warp's, a block's step and several of them
    "t1": dict(lens=[1], D=4, gw=1), "t7": dict(lens=[7, 7], D=8, gw=1), "t9": dict(lens=[9], D=132, gw=1),
    "t63": dict(lens=[63], D=128, gw=1), "t64": dict(lens=[64, 64], D=128, gw=1), "t65": dict(lens=[65], D=256, gw=1),
    "t1000": dict(lens=[1000], D=260, gw=1, xt="f32"), "t2049": dict(lens=[2049, 2049], D=64, gw=1, gt="bf16"),
    # long memory (gates near 1) over many steps
    "memory": dict(lens=[5000], D=36, gw=1, xt="f32", mean=7.0),
    # gates per head: narrow heads, several in a tile, heads that leave lanes idle, wider than a tile, one per row
    "gw4": dict(lens=[130], D=136, gw=4, xt="f32"), "gw32": dict(lens=[130], D=320, gw=32),
    "gw40": dict(lens=[77], D=280, gw=40, gt="bf16"), "gw96": dict(lens=[200], D=288, gw=96),
    "gw120": dict(lens=[129], D=360, gw=120, xt="f32"), "gw128": dict(lens=[70, 70, 70], D=256, gw=128, gt="bf16"),
    "gw132": dict(lens=[100], D=264, gw=132), "gw256": dict(lens=[100], D=512, gw=256, xt="f32"),
    "gw960": dict(lens=[33], D=960, gw=960, gt="bf16"),
    # ragged, with empty sequences first, last and between
    "ragged": dict(lens=[0, 5, 130, 0, 64, 1, 300, 0], D=132, gw=1),
    "ragged_heads": dict(lens=[70, 0, 0, 129, 3], D=384, gw=192, xt="f32"),
    # few channels and many rows (segments), equal and ragged; many sequences (a block each) and fewer (small clusters)
    "segments": dict(lens=[9001], D=12, gw=4, xt="f32"), "segments_bf16": dict(lens=[4200, 4200], D=132, gw=1),
    "segments_ragged": dict(lens=[0, 9000, 3, 0, 13000, 255, 256, 511, 512, 20000], D=8, gw=1, xt="f32", gt="bf16"),
    "segments_wide": dict(lens=[6000], D=320, gw=160, gt="bf16"),
    "blocks": dict(lens=[130] * 240, D=8, gw=1), "blocks_ragged": dict(lens=[3, 200, 70] * 320, D=4, gw=4, xt="f32"),
    "pairs": dict(lens=[300] * 120, D=4, gw=1, gt="bf16"), "fours": dict(lens=[700] * 60, D=8, gw=8),
    "fours_ragged": dict(lens=[1000, 0, 64, 300] * 60, D=4, gw=1, xt="f32"),
    "all_empty": dict(lens=[0, 0], D=8, gw=1),
    # rows further apart than they are long; no states given
    "strided": dict(lens=[100, 100], D=132, gw=1, pad=12), "strided_heads": dict(lens=[9, 100], D=160, gw=40, pad=4, gt="bf16"),
    "no_state": dict(lens=[90], D=132, gw=1, state=False), "no_state_ragged": dict(lens=[90, 0, 2], D=132, gw=12, state=False),
}


@pytest.mark.parametrize("name", list(CASES))
def test_forward_and_backward(name):
    c = case(**CASES[name])
    compare(c, run(c, CASES[name].get("pad", 0)))


def test_gates_of_minus_infinity_start_anew():
    c = case([150, 40], 132, 1, xt="f32")
    c["g"][64, :] = -float("inf")
    c["g"][70, ::3] = -float("inf")
    c["g"][150, :] = -float("inf")   # a sequence's first row: its given state drops out
    compare(c, run(c))
    c = case([150], 256, 64)
    c["g"][64:67] = -float("inf")
    compare(c, run(c))


def test_many_gates_of_zero_and_of_the_lowest_value():
    c = case([300], 64, 1, xt="f32")
    c["g"][:100] = 0.0
    c["g"][100:200:7] = torch.finfo(torch.float32).min
    compare(c, run(c))


def test_nan_and_infinity_stay_in_their_sequence_and_channel():
    c = case([100, 100], 132, 1, xt="f32")
    clean = run(c)
    c["x"][50, 5] = float("nan")
    c["x"][60, 9] = float("inf")
    r = run(c)
    bad = torch.zeros(200, 132, dtype=torch.bool, device="cuda")
    bad[50:100, 5] = True
    bad[60:100, 9] = True
    assert torch.equal(r["y"][~bad], clean["y"][~bad])
    assert bool(torch.isnan(r["y"][50:100, 5]).all()) and bool((r["y"][60:100, 9] == float("inf")).all())
    assert torch.equal(r["dx"], clean["dx"])   # the recurrence is linear in x


def test_gradients_agree_with_differences():
    """The gradients against central differences of the 64-bit forward along random directions: sum y dy + sum hT dhT
    is linear in x and h0; in g the differences of step 1e-4 leave a relative error below 1e-6 (third derivatives of
    exp, gates below 1), the float32 gradients theirs."""
    for gw in (1, 44):
        c = case([70, 0, 129], 132, gw, xt="f32", seed=3)
        r = run(c)
        x, g, h0, dy, dhT = (f64(c[k]) for k in ("x", "g", "h0", "dy", "dhT"))

        def loss(x, g, h0):
            h, _, hT, _ = glr_forward(x, g, c["cuts"], h0, gw)
            return (h * dy).sum() + (hT * dhT).sum()

        rng = np.random.default_rng(1)
        for name, at, grad in (("x", 0, "dx"), ("g", 1, "dg"), ("h0", 2, "dh0")):
            args = [x, g, h0]
            v = rng.standard_normal(args[at].shape)
            lo, hi = list(args), list(args)
            lo[at], hi[at] = args[at] - 1e-4 * v, args[at] + 1e-4 * v
            want = (loss(*hi) - loss(*lo)) / 2e-4
            terms = f64(r[grad]) * v
            assert abs(terms.sum() - want) <= 1e-5 * np.abs(terms).sum(), (gw, name, terms.sum(), want)


def test_two_calls_continue_one():
    """A sequence in two calls, its state handed over in place, is the sequence in one (to rounding: both within the
    bound of the definition), and repeated calls agree bit for bit."""
    c = case([300], 132, 1, xt="f32")
    whole = run(c)
    again = run(c)
    for k in whole:
        assert torch.equal(whole[k], again[k])
    h, he, hT, hTe = glr_forward(f64(c["x"]), f64(c["g"]), c["cuts"], f64(c["h0"]), 1)
    state = c["h0"].clone()
    y = torch.empty_like(c["x"])
    for b, e in ((0, 101), (101, 300)):
        s = sdm.GlrSpec(P=1, rows=e - b, D=132, x_dtype="f32")
        sdm.glr_forward(s, c["x"][b:e], c["g"][b:e], y[b:e], h0=state, hT=state)
    check("y", y, h, he)
    check("hT", state, hT, hTe)


def test_states_in_place_over_segments():
    """hT may be h0 also where a sequence is cut into segments that run at once; dh0 in place of dhT likewise."""
    c = case([9001, 9001], 36, 1, xt="f32")
    want = run(c)
    state = c["h0"].clone()
    states, y, dx, dg = sdm.alloc_glr_states(c["spec"]), *(torch.empty_like(c["x"]) for _ in range(3))
    sdm.glr_forward(c["spec"], c["x"], c["g"], y, h0=state, hT=state, states=states)
    grad = c["dhT"].clone()
    sdm.glr_backward(c["spec"], c["x"], c["g"], c["dy"], states, dx, dg, dhT=grad, dh0=grad)
    for a, b in ((y, "y"), (state, "hT"), (dx, "dx"), (dg, "dg"), (grad, "dh0")):
        assert torch.equal(a, want[b]), b


def test_rows_past_32_bits():
    """More than 2^31 elements: the last sequence's rows lie behind them."""
    P, T, D = 2700, 100, 8192
    spec = sdm.GlrSpec(P=P, rows=P * T, D=D, gate_width=D, x_dtype="bf16", g_dtype="f32")
    x = torch.empty(P * T, D, dtype=torch.bfloat16, device="cuda").normal_()
    g = torch.nn.functional.logsigmoid(torch.empty(P * T, 1, device="cuda").normal_() + 3)
    y, hT, states = torch.empty_like(x), torch.empty(P, D, device="cuda"), sdm.alloc_glr_states(spec)
    sdm.glr_forward(spec, x, g, y, hT=hT, states=states)
    dx, dg = torch.empty_like(x), torch.empty_like(g)
    sdm.glr_backward(spec, x, g, x, states, dx, dg, sdm.alloc_glr_workspace(spec))
    for p in (0, P // 2, P - 1):
        r = slice(p * T, (p + 1) * T)
        cols = slice(D - 40, D)
        xs, gs = f64(x[r]), f64(g[r])
        zero, cuts = np.zeros((1, D)), np.array([0, T])
        h, he, last, laste = glr_forward(xs, gs, cuts, zero, D)
        ddx, ddxe, ddg, ddge, _, _ = glr_backward(xs, gs, cuts, zero, D, xs, zero)
        check("y", y[r, cols], h[:, cols], he[:, cols], torch.bfloat16)
        check("hT", hT[p:p + 1, cols], last[:, cols], laste[:, cols])
        check("dx", dx[r, cols], ddx[:, cols], ddxe[:, cols], torch.bfloat16)
        check("dg", dg[r], ddg, ddge)


def test_many_calls_in_a_row_hand_the_state_on():
    """Kernels are launched as dependents of the one before: 100 chunks and then 50 single tokens back to back, the state
    in place, nothing between the calls."""
    P, D, C, n, m = 3, 516, 40, 100, 50
    c = case([n * C + m] * P, D, 1, xt="f32", seed=8)
    x, g, state = c["x"].view(P, -1, D), c["g"].view(P, -1, D), c["h0"].clone()
    xs = [x[:, i * C:(i + 1) * C].reshape(P * C, D) for i in range(n)] + [x[:, n * C + i].contiguous() for i in range(m)]
    gs = [g[:, i * C:(i + 1) * C].reshape(P * C, D) for i in range(n)] + [g[:, n * C + i].contiguous() for i in range(m)]
    ys = [torch.empty_like(v) for v in xs]
    chunk, one = sdm.GlrSpec(P=P, rows=P * C, D=D, x_dtype="f32"), sdm.GlrSpec(P=P, rows=P, D=D, x_dtype="f32")
    torch.cuda.synchronize()
    for i in range(n):
        sdm.glr_forward(chunk, xs[i], gs[i], ys[i], h0=state, hT=state)
    for i in range(n, n + m):
        sdm.glr_step(one, xs[i], gs[i], state, ys[i])
    h, he, hT, hTe = glr_forward(f64(c["x"]), f64(c["g"]), c["cuts"], f64(c["h0"]), 1)
    y = torch.cat([v.view(P, -1, D) for v in ys], 1)
    check("y", y.view(-1, D), h, he)
    check("state", state, hT, hTe)


def test_offsets_beyond_the_rows_are_cut_and_reported():
    c = case([50, 60], 8, 1, xt="f32")
    c["offsets"] = torch.tensor([0, 50, 400], dtype=torch.int64, device="cuda")
    y, st = torch.zeros_like(c["x"]), torch.zeros(1, dtype=torch.int32, device="cuda")
    sdm.glr_forward(c["spec"], c["x"], c["g"], y, offsets=c["offsets"], h0=c["h0"], status=st)
    assert int(st.item()) == _abi.SDM_DEV_BAD_OFFSET
    h, he, _, _ = glr_forward(f64(c["x"]), f64(c["g"]), c["cuts"], f64(c["h0"]), 1)
    check("y", y, h, he)


@pytest.mark.parametrize("B, D, gw, xt, gt, pad", [
    (1, 4, 1, "f32", "f32", 0), (3, 132, 1, "bf16", "bf16", 8), (64, 256, 64, "bf16", "f32", 0),
    (1000, 120, 120, "f32", "bf16", 4), (5, 960, 12, "bf16", "f32", 0)])
def test_step(B, D, gw, xt, gt, pad):
    """One token per request: three steps in a row equal the recurrence; padding rows and unnamed states stay."""
    gen = torch.Generator().manual_seed(5)
    n = B + 7
    spec = sdm.GlrSpec(P=1, rows=B, D=D, gate_width=gw, x_dtype=xt, g_dtype=gt)
    state = torch.randn(n, D + pad, generator=gen).cuda()[:, :D]
    slots = torch.randperm(n, generator=gen)[:B].to(torch.int32)
    slots[B // 2] = -1 if B > 2 else slots[B // 2]
    want, err = f64(state), np.zeros((n, D))
    live = slots.numpy() >= 0
    idx = slots.numpy()[live]
    for step in range(3):
        x = rows(gen, B, D, xt, pad)
        g = torch.nn.functional.logsigmoid(torch.randn(B, D // gw, generator=gen) + 2.0).to(DT[gt]).cuda()
        y = out(B, D, xt, pad)
        sdm.glr_step(spec, x, g, state, y, slots=slots.cuda())
        a = np.repeat(np.exp(f64(g)), gw, axis=1)[live]
        mag = a * np.abs(want[idx]) + np.abs(f64(x)[live])
        want[idx] = a * want[idx] + f64(x)[live]
        err[idx] = a * err[idx] + 8 * 2.0 ** -24 * mag
        check("y", y[torch.from_numpy(live)], want[idx], err[idx], DT[xt])
        assert bool((y[torch.from_numpy(~live)] == 0).all())
        check("state", state, want, err)


def test_step_without_slots_and_with_a_slot_too_high():
    spec = sdm.GlrSpec(P=1, rows=4, D=8, x_dtype="f32")
    x, g = torch.ones(4, 8, device="cuda"), torch.zeros(4, 8, device="cuda")
    state, y = torch.ones(5, 8, device="cuda"), torch.empty(4, 8, device="cuda")
    sdm.glr_step(spec, x, g, state, y)
    assert bool((state[:4] == 2).all()) and bool((state[4] == 1).all()) and bool((y == 2).all())
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sdm.glr_step(spec, x, g, state, y, slots=torch.tensor([4, 5, -3, 0], dtype=torch.int32, device="cuda"), status=st)
    assert int(st.item()) == _abi.SDM_DEV_BAD_SLOT
    assert state[:, 0].tolist() == [3, 2, 2, 2, 2] and y[:, 0].tolist() == [2, 0, 0, 3]


def test_on_another_stream():
    c = case([500], 132, 1, xt="f32")
    want = run(c)["y"]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = torch.empty_like(c["x"])
    sdm.glr_forward(c["spec"], c["x"], c["g"], y, h0=c["h0"], stream=s)
    s.synchronize()
    assert torch.equal(y, want)


def test_refusals():
    c = case([32], 128, 1, xt="f32")
    s, x, g = c["spec"], c["x"], c["g"]
    y = torch.empty_like(x)
    import dataclasses

    with pytest.raises(ValueError, match="x: expected shape"):
        sdm.glr_forward(s, x[:31], g, y)
    with pytest.raises(TypeError, match="g: expected"):
        sdm.glr_forward(s, x, g.double(), y)
    with pytest.raises(ValueError, match="contiguous"):
        sdm.glr_forward(s, torch.zeros(128, 32, device="cuda").T, g, y)
    with pytest.raises(ValueError, match="overlap"):
        sdm.glr_forward(s, x, g, torch.zeros(1, 128, device="cuda").expand(32, 128))
    with pytest.raises(TypeError, match="GPU only"):
        sdm.glr_forward(s, x.cpu(), g, y)
    with pytest.raises(ValueError, match="states"):
        sdm.glr_backward(s, x, g, x, None, y, torch.empty_like(g))
    with pytest.raises(sdm.SdmError) as e:   # a row 4 bytes off
        sdm.glr_forward(s, torch.zeros(32 * 132, device="cuda")[1:1 + 32 * 128].view(32, 128), g, y)
    assert e.value.status == -4
    with pytest.raises(sdm.SdmError) as e:
        sdm.glr_forward(dataclasses.replace(s, P=3), x, g, y)   # 32 rows are not 3 equal sequences
    assert e.value.status == -2
    wide = case([32], 512, 256, xt="f32")
    with pytest.raises(sdm.SdmError) as e:   # a head wider than a tile needs the workspace
        sdm.glr_backward(wide["spec"], wide["x"], wide["g"], wide["dy"], sdm.alloc_glr_states(wide["spec"]),
                         torch.empty_like(wide["x"]), torch.empty_like(wide["g"]))
    assert e.value.status == -5
