"""The embedding (sdm_embed, sdm_embed_backward) against its definition in 64 bits: a row is one product (u = 2^-24), a row of the
gradient a sum of n products in any order (n + 2 u of the sum of their magnitudes)."""

import numpy as np
import pytest
import torch

import sparse_slot_memory_gb300 as sdm
from operators_testlib import U, check, f64
from sparse_slot_memory_gb300 import _abi

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def case(T, V, D, tt="f32", xt="bf16", pad=0, skew=0.0, ids=None, seed=0):
    gen = torch.Generator().manual_seed(seed)

    def wide(n, t, scale=1.0):
        x = torch.full((n, D + pad), float("nan"))
        x[:, :D] = torch.randn(n, D, generator=gen) * scale
        return x.to(DT[t]).cuda()[:, :D]

    if ids is None:
        u = torch.rand(T, generator=gen)
        ids = (u ** (1 + skew) * V).long().clamp(0, V - 1)
        ids[::17] = -1
    s = sdm.EmbedSpec(tokens=T, V=V, D=D, table_dtype=tt, dtype=xt, scale=1.7)
    return s, {"ids": ids.to(torch.int32).cuda(), "table": wide(V, tt), "dy": wide(T, xt)}


def compare(s, c, pad=0, accumulate=False):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = torch.full((s.tokens, s.D + pad), float("nan"), dtype=DT[s.dtype], device="cuda")[:, :s.D]
    sdm.embed(s, c["ids"], c["table"], y, status=st)
    ids, table, dy = f64(c["ids"]).astype(int), f64(c["table"]), f64(c["dy"])
    real = (ids >= 0) & (ids < s.V)
    scale = float(np.float32(s.scale))
    want = np.where(real[:, None], scale * table[np.where(real, ids, 0)], 0.0)
    check("y", y, want, U * np.abs(want), DT[s.dtype])
    d = torch.full((s.V, s.D + pad), float("nan"), dtype=DT[s.table_dtype], device="cuda")[:, :s.D]
    base = np.zeros((s.V, s.D))
    if accumulate:
        d.copy_(torch.randn(s.V, s.D))
        base = f64(d)
    ws = sdm.alloc_embed_workspace(s)
    ws.fill_(255)
    sdm.embed_backward(s, c["ids"], c["dy"], d, ws, accumulate=accumulate, status=st)
    want, mag, n = np.zeros((s.V, s.D)), np.zeros((s.V, s.D)), np.zeros((s.V, 1))
    np.add.at(want, ids[real], scale * dy[real])
    np.add.at(mag, ids[real], scale * np.abs(dy[real]))
    np.add.at(n, ids[real], 1)
    tol = (n + 2) * U * mag + 2 * U * np.abs(base) * (n > 0)
    if accumulate:   # rows without tokens are not touched
        assert np.array_equal(f64(d)[n[:, 0] == 0], base[n[:, 0] == 0])
    check("dtable", d, base + want, tol, DT[s.table_dtype])
    return int(st.item()), y, d


CASES = {
    "one": dict(T=1, V=1, D=4), "few": dict(T=5, V=300, D=8, tt="bf16"), "t0": dict(T=0, V=10, D=16), "d36": dict(T=300, V=70, D=36, xt="f32"),
    # one pass of the sort, two, three; ids at the digits' borders
    "v255": dict(T=1000, V=255, D=64), "v256": dict(T=1000, V=256, D=64, tt="bf16", xt="f32"), "v65535": dict(T=3000, V=65535, D=16),
    "v65536": dict(T=3000, V=65536, D=16, tt="bf16"), "v100000": dict(T=9000, V=100000, D=20, xt="f32"),
    # columns on both sides of a warp's slice; many tokens for few rows
    "d512": dict(T=700, V=40, D=512), "d516": dict(T=700, V=40, D=516, xt="f32"), "d1000": dict(T=2000, V=1000, D=1000, skew=4.0),
    "d2052": dict(T=500, V=9, D=2052, tt="bf16"), "hot": dict(T=20000, V=50, D=132, skew=9.0), "strided": dict(T=400, V=90, D=132, pad=8),
    "strided_f32": dict(T=400, V=90, D=40, pad=4, xt="f32", tt="bf16"),
}


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("name", list(CASES))
def test_rows_and_gradient(name, accumulate):
    s, c = case(**CASES[name])
    assert compare(s, c, CASES[name].get("pad", 0), accumulate)[0] == 0


def test_counts_around_the_block_s_rows():
    """Rows of no, one and several tokens around a part of 16 and a block of parts, and of 5000, in a mixed order."""
    counts = [0, 1, 3, 4, 5, 15, 16, 17, 32, 33, 128, 129, 5000, 1025]
    ids = torch.cat([torch.full((n,), i) for i, n in enumerate(counts)])
    ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(1))]
    for xt in ("bf16", "f32"):
        s, c = case(len(ids), len(counts) + 2, 260, xt=xt, ids=ids)
        assert compare(s, c)[0] == 0


def test_every_token_the_same_and_every_token_padding():
    s, c = case(3000, 20, 64, ids=torch.full((3000,), 7))
    assert compare(s, c)[0] == 0
    s, c = case(300, 20, 64, ids=torch.full((300,), -5))
    st, y, d = compare(s, c)
    assert st == 0 and bool((y == 0).all()) and bool((d == 0).all())


def test_ids_behind_the_table_are_padding_and_reported():
    ids = torch.tensor([0, 5, 19, 20, 2 ** 31 - 1, -2 ** 31, -1, 5])
    s, c = case(8, 20, 64, ids=ids)
    assert compare(s, c)[0] == _abi.SDM_DEV_BAD_TOKEN


def test_infinity_and_nan_stay_in_their_rows():
    s, c = case(500, 60, 64, xt="f32")
    ids = f64(c["ids"]).astype(int)
    c["dy"][3, 5] = float("inf")
    c["dy"][40, 7] = float("nan")
    d = torch.empty(60, 64, device="cuda")
    sdm.embed_backward(s, c["ids"], c["dy"], d, sdm.alloc_embed_workspace(s))
    bad = torch.zeros(60, 64, dtype=torch.bool)
    bad[ids[3], 5] = bad[ids[40], 7] = True
    assert torch.equal(~d.isfinite().cpu(), bad)


def test_padding_takes_nothing_from_its_row():
    """A padding token's dy may hold anything."""
    s, c = case(300, 30, 64, xt="f32")
    c["dy"][c["ids"] < 0] = float("nan")
    d = torch.empty(30, 64, device="cuda")
    sdm.embed_backward(s, c["ids"], c["dy"], d, sdm.alloc_embed_workspace(s))
    assert bool(d.isfinite().all())


def test_runs_are_bitwise_equal_and_follow_the_tokens_order():
    s, c = case(20000, 300, 132, skew=6.0, xt="f32")
    out = []
    for _ in range(3):
        d = torch.empty(300, 132, device="cuda")
        sdm.embed_backward(s, c["ids"], c["dy"], d, sdm.alloc_embed_workspace(s))
        out.append(d)
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])
    # rows of up to 16 tokens are added in the tokens' order
    ids = c["ids"].long()
    for v in [int(i) for i in range(300) if 1 < int((ids == i).sum()) <= 16][:20]:
        t = torch.zeros(132, device="cuda")
        for i in torch.nonzero(ids == v).reshape(-1).tolist():
            t = t + c["dy"][i]
        assert torch.equal(out[0][v], t * s.scale)


def test_more_than_2_31_elements():
    V, D = 1 << 18, 10240
    s = sdm.EmbedSpec(tokens=6, V=V, D=D, table_dtype="bf16", dtype="bf16")
    table = torch.empty(V, D, dtype=torch.bfloat16, device="cuda").normal_()
    ids = torch.tensor([V - 1, 0, V - 3, V - 1, 209716, 7], dtype=torch.int32, device="cuda")
    y = torch.empty(6, D, dtype=torch.bfloat16, device="cuda")
    sdm.embed(s, ids, table, y)
    assert torch.equal(y, table[ids.long()])
    table.fill_(float("nan"))
    sdm.embed_backward(s, ids, y, table, sdm.alloc_embed_workspace(s))
    assert torch.equal(table[V - 3], y[2]) and torch.equal(table[209716], y[4]) and torch.equal(table[V - 1], (y[0].float() + y[3].float()).bfloat16())
    assert bool((table[V - 2] == 0).all()) and not bool(table[::1009].isnan().any())
