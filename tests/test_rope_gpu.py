"""Norms of query and key heads with the position rotation (sdm_qk_norm_rope, its backward, sdm_rope_table) against
their definition in 64 bits (tests/operators_testlib.py, which derives the bounds)."""

import math

import numpy as np
import pytest
import torch

import sparse_slot_memory_gb300 as sdm
from operators_testlib import U, check, f64, rope_head
from sparse_slot_memory_gb300 import _abi

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def case(T, Hq, Hk, hd, rd, layout="half", dtype="bf16", norm=True, weights=True, pad=0, max_pos=500, eps=1e-6, seed=0):
    gen = torch.Generator().manual_seed(seed)
    spec = sdm.RopeSpec(tokens=T, q_heads=Hq, k_heads=Hk, hd=hd, rot_dim=rd, max_pos=max_pos, layout=layout, dtype=dtype,
                        norm=norm, eps=eps)
    c = {"spec": spec}
    # queries, keys and `pad` more columns in one row, as a fused projection gives them
    row = (torch.randn(T, (Hq + Hk) * hd + pad, generator=gen) * 2).to(DT[dtype]).cuda()
    c["q"] = row[:, :Hq * hd].view(T, Hq, hd) if Hq else None
    c["k"] = row[:, Hq * hd:(Hq + Hk) * hd].view(T, Hk, hd) if Hk else None
    for n, H in (("dq_out", Hq), ("dk_out", Hk)):
        c[n] = torch.randn(T, H, hd, generator=gen).to(DT[dtype]).cuda()
    c["wq"] = (1 + 0.2 * torch.randn(hd, generator=gen)).cuda() if weights else None
    c["wk"] = (1 + 0.2 * torch.randn(hd, generator=gen)).cuda() if weights else None
    pos = torch.randint(0, max_pos, (T,), generator=gen)
    if T > 3:
        pos[2] = -1      # a padding token
        pos[T // 2] = 0
    c["pos"] = pos.to(torch.int32).cuda()
    c["table"] = torch.randn(max_pos, max(rd, 1), generator=gen).cuda()[:, :rd].contiguous()
    return c


def run(c):
    s = c["spec"]
    r = {}
    for n, H in (("q_out", s.q_heads), ("k_out", s.k_heads), ("dq", s.q_heads), ("dk", s.k_heads)):
        r[n] = torch.full((s.tokens, H, s.hd), float("nan"), dtype=DT[s.dtype], device="cuda")
    r["dwq"], r["dwk"] = (torch.full((s.hd,), float("nan"), device="cuda") for _ in range(2))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sdm.qk_norm_rope(s, c["q"], c["k"], c["pos"], c["table"], c["wq"], c["wk"], r["q_out"], r["k_out"], status=st)
    sdm.qk_norm_rope_backward(s, c["dq_out"], c["dk_out"], c["q"], c["k"], c["pos"], c["table"], c["wq"], c["wk"], r["dq"],
                              r["dk"], r["dwq"], r["dwk"], sdm.alloc_rope_workspace(s), status=st)
    assert int(st.item()) == 0
    return r


def compare(c, r):
    s = c["spec"]
    pos, table = c["pos"].cpu().numpy(), f64(c["table"])
    for kind, H in (("q", s.q_heads), ("k", s.k_heads)):
        if not H:
            continue
        w = f64(c["w" + kind]) if c["w" + kind] is not None else None
        o, oe, dx, dxe, dw, dwe = rope_head(f64(c[kind]), w, pos, table, s.rot_dim, s.layout, s.norm, np.float32(s.eps),
                                            f64(c[f"d{kind}_out"]))
        check(kind + "_out", r[kind + "_out"], o, oe, DT[s.dtype])
        check("d" + kind, r["d" + kind], dx, dxe, DT[s.dtype])
        if s.norm:
            check("dw" + kind, r["dw" + kind], dw, dwe)


CASES = {
    "one": dict(T=1, Hq=1, Hk=1, hd=8, rd=8), "hd64": dict(T=33, Hq=3, Hk=1, hd=64, rd=64),
    "hd128": dict(T=70, Hq=8, Hk=2, hd=128, rd=128), "hd128_f32": dict(T=21, Hq=4, Hk=4, hd=128, rd=128, dtype="f32"),
    "inter": dict(T=40, Hq=4, Hk=1, hd=128, rd=128, layout="interleaved"),
    "inter_part": dict(T=40, Hq=5, Hk=2, hd=64, rd=32, layout="interleaved", dtype="f32"),
    "part": dict(T=40, Hq=4, Hk=2, hd=96, rd=40), "hd120": dict(T=300, Hq=6, Hk=1, hd=120, rd=64),
    "hd136": dict(T=9, Hq=2, Hk=3, hd=136, rd=136), "hd256": dict(T=17, Hq=2, Hk=2, hd=256, rd=64, dtype="f32"),
    "hd512": dict(T=5, Hq=2, Hk=1, hd=512, rd=512, layout="interleaved"),
    "hd960": dict(T=5, Hq=1, Hk=2, hd=960, rd=960), "hd1024": dict(T=3, Hq=1, Hk=1, hd=1024, rd=8, dtype="f32"),
    "norm_only": dict(T=30, Hq=2, Hk=2, hd=64, rd=0), "turn_only": dict(T=30, Hq=2, Hk=2, hd=64, rd=48, norm=False),
    "no_weights": dict(T=30, Hq=2, Hk=2, hd=128, rd=128, weights=False),
    "no_keys": dict(T=30, Hq=3, Hk=0, hd=64, rd=64), "no_queries": dict(T=30, Hq=0, Hk=3, hd=64, rd=64),
    "strided": dict(T=50, Hq=4, Hk=2, hd=64, rd=64, pad=68), "many": dict(T=3000, Hq=4, Hk=2, hd=128, rd=64),
    "eps": dict(T=30, Hq=2, Hk=2, hd=64, rd=64, eps=0.5, dtype="f32"),
}


@pytest.mark.parametrize("name", list(CASES))
def test_forward_and_backward(name):
    c = case(**CASES[name])
    compare(c, run(c))


def test_zero_rows_have_finite_results():
    c = case(8, 2, 2, 64, 64, dtype="f32")
    c["q"].zero_()
    r = run(c)
    compare(c, r)
    assert bool((r["q_out"] == 0).all()) and bool(torch.isfinite(r["dq"]).all())


def test_rotation_alone_does_not_look_at_the_inputs_in_its_backward():
    c = case(30, 3, 1, 64, 48, norm=False)
    want = run(c)
    c["q"][5, 1, 3], c["k"][9] = float("nan"), float("inf")
    r = run(c)
    assert torch.equal(r["dq"], want["dq"]) and torch.equal(r["dk"], want["dk"])
    assert bool(torch.isnan(r["q_out"][5, 1]).any()) and torch.equal(r["q_out"][5, 2], want["q_out"][5, 2])


def test_in_place_and_repeated_calls():
    c = case(70, 8, 2, 128, 64, dtype="bf16", pad=8)
    s, want = c["spec"], run(c)
    again = run(c)
    for k in want:
        assert torch.equal(want[k], again[k]), k
    q, k = c["q"].clone(), c["k"].clone()
    # gradients over the outputs' gradients, then the forward over its inputs
    gq, gk = c["dq_out"].clone(), c["dk_out"].clone()
    sdm.qk_norm_rope_backward(s, gq, gk, q, k, c["pos"], c["table"], c["wq"], c["wk"], gq, gk)
    sdm.qk_norm_rope(s, q, k, c["pos"], c["table"], c["wq"], c["wk"], q, k)
    for a, b in ((q, "q_out"), (k, "k_out"), (gq, "dq"), (gk, "dk")):
        assert torch.equal(a, want[b]), b


def test_positions_beyond_the_table_are_padding_and_reported():
    c = case(20, 2, 1, 64, 64, dtype="f32", max_pos=100)
    c["pos"][5] = 100
    c["pos"][6] = 2 ** 31 - 1
    s = c["spec"]
    q, k = torch.empty_like(c["dq_out"]), torch.empty_like(c["dk_out"])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sdm.qk_norm_rope(s, c["q"], c["k"], c["pos"], c["table"], c["wq"], c["wk"], q, k, status=st)
    assert int(st.item()) == _abi.SDM_DEV_BAD_POSITION
    assert bool((q[5:7] == 0).all()) and bool((k[5:7] == 0).all()) and bool((q[7] != 0).any())


def test_gradients_agree_with_differences():
    """Against central differences of the 64-bit forward along random directions (step 1e-5: a relative error below
    1e-7 for these smooth functions; the float32 gradients theirs)."""
    c = case(12, 3, 2, 64, 40, dtype="f32", layout="interleaved")
    s, r = c["spec"], run(c)
    pos, table = c["pos"].cpu().numpy(), f64(c["table"])
    rng = np.random.default_rng(2)
    for kind in "qk":
        x, w, d = f64(c[kind]), f64(c["w" + kind]), f64(c[f"d{kind}_out"])
        loss = lambda x, w: (rope_head(x, w, pos, table, s.rot_dim, s.layout, True, 1e-6)[0] * d).sum()
        v, vw = rng.standard_normal(x.shape), rng.standard_normal(w.shape)
        for want, terms in (((loss(x + 1e-5 * v, w) - loss(x - 1e-5 * v, w)) / 2e-5, f64(r["d" + kind]) * v),
                            ((loss(x, w + 1e-5 * vw) - loss(x, w - 1e-5 * vw)) / 2e-5, f64(r["dw" + kind]) * vw)):
            assert abs(terms.sum() - want) <= 1e-5 * np.abs(terms).sum(), kind


def test_no_tokens():
    c = case(0, 2, 2, 64, 64)
    r = run(c)
    assert bool((r["dwq"] == 0).all()) and bool((r["dwk"] == 0).all())


@pytest.mark.parametrize("scaling", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0),
                                     dict(scaling="by_parts", factor=4.0, trained_len=4096, low=1.0, high=32.0)])
def test_table(scaling):
    """cos and sin of position times angle for positions up to 2^20, scaled frequencies: the reduction is exact, so the
    error is that of float32 half turns (2^-25 of a half turn, times pi), sincospif's 2 ulp and one product."""
    rd, n = 64, 1 << 20
    spec = sdm.RopeSpec(tokens=1, q_heads=1, k_heads=1, hd=64, rot_dim=rd, max_pos=n)
    f = sdm.rope_frequencies(rd, base=500000.0, **scaling)
    table = torch.full((n, rd), float("nan"), device="cuda")
    sdm.rope_table(spec, f, table, scale=1.25)
    pos = np.unique(np.concatenate([np.arange(70), np.arange(n - 70, n), np.random.default_rng(0).integers(0, n, 3000)]))
    got = f64(table[torch.from_numpy(pos).cuda()])
    # whole turns drop out in integers here too: the angle of one position as a fraction of 2^-60 turns
    turn = np.array([int(round(math.ldexp(v / (2 * math.pi), 60))) for v in f], dtype=object)
    frac = ((pos.astype(object)[:, None] * turn[None, :]) % (1 << 60)).astype(np.float64) / 2.0 ** 60 * 2 * math.pi
    want = 1.25 * np.concatenate([np.cos(frac), np.sin(frac)], 1)
    # 2^-60 turns and the double's own rounding of the angle, a million positions on, and the float32 steps above
    tol = 1.25 * (n * 2 * math.pi * (2.0 ** -60 + 2.0 ** -54) + 2 * U * math.pi + 8 * U)
    assert np.abs(got - want).max() <= tol


def test_frequencies():
    base = sdm.rope_frequencies(8)
    assert np.allclose(base, [1.0, 0.1, 0.01, 0.001], rtol=1e-12)
    assert np.allclose(sdm.rope_frequencies(8, scaling="linear", factor=4), np.array(base) / 4, rtol=1e-12)
    b = sdm.rope_frequencies(8, scaling="base", factor=4)
    assert b[0] == 1.0 and math.isclose(b[-1], base[-1] / 4, rel_tol=1e-12)
    p = sdm.rope_frequencies(64, scaling="by_parts", factor=4, trained_len=4096, low=1, high=32)
    q = sdm.rope_frequencies(64)
    turns = [4096 * v / (2 * math.pi) for v in q]
    for a, v, t in zip(p, q, turns):
        assert (a == v) if t >= 32 else math.isclose(a, v / 4, rel_tol=1e-12) if t <= 1 else v / 4 < a < v
    with pytest.raises(ValueError):
        sdm.rope_frequencies(64, scaling="by_parts", factor=4)
    with pytest.raises(ValueError):
        sdm.rope_frequencies(64, scaling="other")


def test_refusals():
    c = case(8, 2, 1, 64, 64)
    s, q, k = c["spec"], c["dq_out"].clone(), c["dk_out"].clone()
    args = (c["pos"], c["table"], c["wq"], c["wk"], q, k)
    import dataclasses

    with pytest.raises(ValueError, match="q: expected shape"):
        sdm.qk_norm_rope(s, c["q"][:, :1], c["k"], *args)
    with pytest.raises(ValueError, match="table: expected at least"):
        sdm.qk_norm_rope(s, c["q"], c["k"], c["pos"], c["table"][:10].contiguous(), c["wq"], c["wk"], q, k)
    with pytest.raises(TypeError, match="positions"):
        sdm.qk_norm_rope(s, c["q"], c["k"], c["pos"].long(), *args[1:])
    for bad, code in ((dict(hd=68), -4), (dict(rot_dim=12), -4), (dict(rot_dim=72), -2), (dict(max_pos=0), -2),
                      (dict(eps=-1.0), -2), (dict(hd=1032), -2)):
        t = dataclasses.replace(s, **bad)
        st = _abi.load().sdm_qk_norm_rope(t.c(), q.data_ptr(), 128, k.data_ptr(), 64, c["pos"].data_ptr(),
                                          c["table"].data_ptr(), None, None, q.data_ptr(), 128, k.data_ptr(), 64, None, None)
        assert st == code, bad
    with pytest.raises(sdm.SdmError) as e:   # the weights' gradients need the workspace
        sdm.qk_norm_rope_backward(s, q, k, c["q"], c["k"], *args[:4], q, k, torch.empty(64, device="cuda"))
    assert e.value.status == -5
    off = torch.zeros(8 * 128 + 2, dtype=torch.bfloat16, device="cuda")[2:].view(8, 2, 64)
    with pytest.raises(sdm.SdmError) as e:
        sdm.qk_norm_rope(s, off, c["k"], *args)
    assert e.value.status == -4
