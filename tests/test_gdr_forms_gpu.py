"""The gated delta rule in the forms that sizes choose (value columns of a block, boxes or copies by hand), with rows that repeat, far
apart in memory, and on tensors past 2^31 elements."""

import pytest
import torch

import sparse_slot_memory_gb300 as sdm
from test_gdr_gpu import case, compare, run

pytestmark = pytest.mark.gpu


FORMS = {
    # more sequences and heads than SMs: blocks of 64 and 128 columns, whole blocks and tails, keys of 64 and 128
    "many_128": dict(lens=[70] * 20, Hk=2, Hv=8, dk=128, dv=128), "many_64": dict(lens=[64, 1, 65, 130] * 10, Hv=4, Hk=1, dk=64, dv=128),
    "one_round": dict(lens=[130] * 38, Hk=2, Hv=4, dk=128, dv=128), "one_round_64": dict(lens=[129, 64] * 19, Hv=4, dk=64, dv=128),
    # heads that boxes do not serve, beside the same with
    "columns_96": dict(lens=[130] * 20, Hv=8, dk=64, dv=96), "columns_64": dict(lens=[200, 64], Hv=2, dk=128, dv=64),
    "columns_32": dict(lens=[200, 64], Hv=2, dk=128, dv=32), "columns_16": dict(lens=[128], Hv=2, dk=64, dv=16),
    "keys_112": dict(lens=[192], Hv=2, dk=112, dv=128), "keys_64": dict(lens=[192], Hk=2, Hv=2, dk=64, dv=64, gt="bf16"),
    # fewer rows than a box has
    "rows_63": dict(lens=[63], dk=128, dv=128), "rows_40": dict(lens=[10, 30], dk=64, dv=64),
    # several blocks of each head in turn on one SM
    "units": dict(lens=[450, 64, 3], Hk=8, Hv=32, dk=64, dv=64),
}


@pytest.mark.parametrize("name", list(FORMS))
def test_forms(name):
    c = case(**FORMS[name])
    compare(c, run(c))


SEGMENTS = {
    # few heads of long sequences, whose rows are walked in segments: boxes and copies by hand, tails, a sequence of fewer blocks than
    # segments and none, blocks of other sequences' lengths
    "boxes": dict(lens=[4160], Hk=1, Hv=2, dk=64, dv=128), "wide": dict(lens=[4096], dk=128, dv=64), "narrow": dict(lens=[4131], Hk=1, Hv=2, dk=24, dv=40),
    "ragged": dict(lens=[3, 9000, 0, 7500, 130], dk=64, dv=64), "no_state": dict(lens=[8300], dk=32, dv=32, state=False, gt="bf16"),
    "slow": dict(lens=[4200], dk=64, dv=64, rate=0.003), "outside": dict(lens=[5000], dk=16, dv=8, before=70, behind=9),
}


@pytest.mark.parametrize("name", list(SEGMENTS))
def test_segments(name):
    c = case(**SEGMENTS[name])
    compare(c, run(c), whole=False)


def test_segments_with_states_in_place_and_gates_that_start_anew():
    c = case([4400], Hv=2, dk=64, dv=64)
    c["g"][700:710, 0] = -float("inf")
    c["g"][2111, :] = -float("inf")
    want = run(c, False)
    compare(c, want, False, whole=False)
    h, y, s = c["h0"].clone(), torch.empty_like(c["v"]), c["spec"]
    sdm.gdr_forward(s, *[c[n] for n in ("q", "k", "v", "g", "beta")], y, sdm.alloc_gdr_workspace(s, backward=False), h0=h, hT=h)
    assert torch.equal(h, want["hT"]) and torch.equal(y, want["y"])


def test_segments_keep_what_is_before_a_nan():
    """A value that is not finite spoils what follows it, across segments, and nothing before its block nor another head's."""
    c = case([4400], Hk=2, Hv=2, dk=64, dv=64)
    want = run(c, False)
    for name, at in (("v", 2500), ("k", 2500)):
        d = dict(c) | {name: c[name].clone()}
        d[name][at, 0, 3] = float("nan")
        got = run(d, False)
        block = at // 64 * 64
        assert torch.equal(got["y"][:block], want["y"][:block]) and torch.equal(got["y"][:, 1], want["y"][:, 1])
        assert torch.equal(got["hT"][:, 1], want["hT"][:, 1])
        assert bool(got["y"][at + 64:, 0].isnan().any(1).all()) and bool(got["hT"][0, 0].isnan().any())


@pytest.mark.parametrize("xt", ["bf16", "f32"])
def test_rows_that_repeat(xt):
    """Inputs with a distance of 0 between rows are one row for all."""
    c = case([150, 64], Hk=1, Hv=2, dk=64, dv=64, xt=xt)
    for n in ("q", "v", "g"):
        c[n] = c[n][:1].expand(c["spec"].rows, *c[n].shape[1:])
    plain = dict(c) | {n: c[n].contiguous() for n in ("q", "v", "g")}
    compare(c, run(c))
    a, b = run(c), run(plain)
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_heads_of_one_projection():
    """Queries, keys and values as columns of one projection's rows, gates as columns of another's."""
    c = case([200, 70, 64], Hk=2, Hv=4, dk=64, dv=128)
    n = c["spec"].rows
    wide = torch.full((n, 2 * 2 * 64 + 2 * 4 * 128 + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    gates = torch.full((n, 9), float("nan"), device="cuda")
    views, at = dict(c), 8
    for name, H, d in (("k", 2, 64), ("v", 4, 128), ("q", 2, 64), ("dy", 4, 128)):
        views[name] = wide[:, at:at + H * d].unflatten(1, (H, d))
        views[name].copy_(c[name])
        at += H * d
    for i, name in enumerate(("beta", "g")):
        views[name] = gates[:, 1 + 4 * i:5 + 4 * i]
        views[name].copy_(c[name])
    a, b = run(c), run(views)
    assert all(torch.equal(a[x], b[x]) for x in a)


@pytest.mark.parametrize("xt", ["bf16", "f32"])
def test_past_2_31_elements(xt):
    """Rows whose elements lie up to 2.3e9 elements from the first: the answers of the last of many sequences are those of its own."""
    ld, tail = 32768 if xt == "bf16" else 16384, 200
    rows = 70000 if xt == "bf16" else 140000
    c = case([tail], Hk=1, Hv=2, dk=64, dv=64, xt=xt, state=False)
    dt = c["q"].dtype
    big = torch.zeros(rows, ld, dtype=dt, device="cuda")
    names = (("q", 1), ("k", 1), ("v", 2), ("dy", 2), ("y", 2), ("dq", 1), ("dk", 1), ("dv", 2))
    view, at = {}, 0
    for name, H in names:
        view[name] = big[:, at:at + H * 64].unflatten(1, (H, 64))
        at += H * 64
    gates = torch.zeros(4, rows, 2, device="cuda")
    view |= {"g": gates[0], "beta": gates[1], "dg": gates[2], "dbeta": gates[3]}
    for name in ("q", "k", "v", "dy", "g", "beta"):
        view[name][rows - tail:].copy_(c[name])
    s = sdm.GdrSpec(P=2, rows=rows, k_heads=1, v_heads=2, dk=64, dv=64, x_dtype=xt, scale=c["spec"].scale)
    offsets = torch.tensor([rows - tail - 1, rows - tail, rows], device="cuda")
    states, ws = sdm.alloc_gdr_states(s), sdm.alloc_gdr_workspace(s)
    x = [view[n] for n in ("q", "k", "v", "g", "beta")]
    sdm.gdr_forward(s, *x, view["y"], ws, offsets=offsets, states=states)
    sdm.gdr_backward(s, *x, view["dy"], states, *[view[n] for n in ("dq", "dk", "dv", "dg", "dbeta")], ws, offsets=offsets)
    got = {n: view[n] for n in ("y", "dq", "dk", "dv", "dg", "dbeta")}
    compare(c, {n: t[rows - tail:] for n, t in got.items()}, whole=False)   # in segments, as the rows of all sequences suggest them
    for n, t in got.items():
        assert not t[:rows - tail].any(), n


def test_step_of_a_table_past_2_31_elements():
    Hv, d, slots = 16, 128, 9000   # 2.36e9 elements
    s = sdm.GdrSpec(P=1, rows=2, k_heads=Hv, v_heads=Hv, dk=d, dv=d)
    state = torch.empty(slots, Hv, d, d, device="cuda")
    gen = torch.Generator().manual_seed(0)
    r = lambda *shape: torch.randn(*shape, generator=gen).cuda()
    x = [r(2, Hv, d).bfloat16() for _ in range(3)] + [-r(2, Hv).abs(), r(2, Hv).sigmoid()]
    small = r(2, Hv, d, d)
    state[0], state[slots - 1] = small[0], small[1]
    y, z = torch.empty(2, Hv, d, dtype=torch.bfloat16, device="cuda"), torch.empty(2, Hv, d, dtype=torch.bfloat16, device="cuda")
    sdm.gdr_step(s, *x, state, y, slots=torch.tensor([0, slots - 1], dtype=torch.int32, device="cuda"))
    sdm.gdr_step(s, *x, small, z)
    assert torch.equal(y, z) and torch.equal(state[0], small[0]) and torch.equal(state[slots - 1], small[1])
