"""A value that is not finite stays with its sequence and head, forward and backward, where blocks of many heads and sequences follow
one another on an SM."""

import pytest
import torch

from test_gdr_gpu import case, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("name", ["v", "q", "k", "dy", "g", "beta", "h0", "dhT"])
@pytest.mark.parametrize("xt, Hk, Hv, dk, dv", [("bf16", 8, 32, 64, 64), ("bf16", 4, 8, 128, 128), ("f32", 2, 4, 72, 40)])
def test_stays_with_its_sequence_and_head(xt, Hk, Hv, dk, dv, name, value):
    lens = [450, 64, 300, 3]
    c = case(lens, Hk=Hk, Hv=Hv, dk=dk, dv=dv, xt=xt)
    clean = run(c)
    R, p, rows = Hv // Hk, 2, slice(514, 814)
    d = dict(c) | {name: c[name].clone()}
    key = 1   # the key head whose value heads may have it
    if name in ("h0", "dhT"):
        d[name][p, key * R, 3, 5] = value
    elif name in ("g", "beta"):
        d[name][600, key * R] = value
    else:
        d[name][600, key if name in ("q", "k") else key * R, 3] = value
    r = run(d)
    spoiled = False
    for n in r:
        mine = torch.zeros(r[n].shape[:2], dtype=torch.bool)
        heads = slice(key, key + 1) if n in ("dq", "dk") else slice(key * R, (key + 1) * R)
        mine[p if n in ("hT", "dh0") else rows, heads] = True
        mine = mine.cuda()
        assert torch.equal(r[n][~mine], clean[n][~mine]), n
        spoiled |= not bool(r[n][mine].isfinite().all())
    assert spoiled
