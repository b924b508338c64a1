"""Corners of the token log probabilities: masked logits at other scales and under large gradients of the entropy, and finite
logits whose products leave float32's range, and the gradient in the logits' place. The values are those of
tests/operators_testlib.py in 64 bits, with its bounds."""

import numpy as np
import pytest
import torch

import sparse_slot_memory_gb300 as sdm
from operators_testlib import check, f64, logprobs, logprobs_backward, order_topk

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def run(x, t, scale, K=0, dh=1.0, seed=9):
    """Forward and backward of logits x [N, V]; the entropies' gradients are `dh` times N(0, 1)."""
    N, V = x.shape
    s = sdm.LogprobSpec(rows=N, V=V, K=K, dtype="bf16" if x.dtype == torch.bfloat16 else "f32", scale=scale)
    gen = torch.Generator().manual_seed(seed)
    r = {k: torch.full((N,), float("nan"), device="cuda") for k in ("logp", "entropy", "lse")}
    r["top_vals"] = torch.full((N, K), float("nan"), device="cuda")
    r["top_idx"] = torch.full((N, K), -7, dtype=torch.int32, device="cuda")
    r["d_logp"], r["d_entropy"] = torch.randn(N, generator=gen).cuda(), (dh * torch.randn(N, generator=gen)).cuda()
    r["dlogits"] = torch.full((N, V), float("nan"), dtype=x.dtype, device="cuda")
    sdm.token_logprobs(s, x, t, r["logp"], r["entropy"], r["lse"], r["top_vals"], r["top_idx"])
    sdm.token_logprobs_backward(s, x, t, r["lse"], r["entropy"], r["d_logp"], r["dlogits"], r["d_entropy"])
    return r


def compare(x, t, scale, r, K=0):
    """Against the definition; past float32's range log probabilities are -inf, and a finite lse its last finite values."""
    X, tt, sc = f64(x), t.cpu().numpy(), float(np.float32(scale))
    with np.errstate(over="ignore"):
        f = logprobs(X, tt, sc)
        stored = lambda v: v.astype(np.float32).astype(np.float64)
        check("logp", r["logp"], stored(f["logp"]), f["logp_e"])
        check("entropy", r["entropy"], f["H"], f["H_e"])
        top = float(np.finfo(np.float32).max)
        check("lse", r["lse"], np.where(np.isinf(f["lse"]), f["lse"], f["lse"].clip(-top, top)), f["lse_e"])
        if K:
            top = order_topk(X, K)
            assert np.array_equal(r["top_idx"].cpu().numpy(), top)
            at = (np.arange(len(X))[:, None], top)
            check("top_vals", r["top_vals"], stored(f["logs"][at]), f["logs_e"][at])
    d, e = logprobs_backward(X, tt, sc, f64(r["d_logp"]), f64(r["d_entropy"]))
    check("dlogits", r["dlogits"], d, e, x.dtype)


def masked(N, V, dtype, scale, seed=0):
    """Logits of N(0, 4) behind the scale, a third of them -inf, a third the type's lowest value."""
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(N, V, generator=gen) * (2.0 / scale)).to(DT[dtype])
    u = torch.rand(N, V, generator=gen)
    x[u < 1 / 3] = -float("inf")
    x[u > 2 / 3] = torch.finfo(DT[dtype]).min
    t = torch.randint(0, V, (N,), generator=gen).to(torch.int32)
    for i in range(N):   # a target that is left, but for the last row's, whose probability is 0
        t[i] = torch.nonzero((u[i] >= 1 / 3) & (u[i] <= 2 / 3))[int(t[i]) % 10] if i + 1 < N else t[i]
    return x.cuda(), t.cuda()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("scale, dh", [(0.01, 1e5), (1.0, 1e9), (10.0, 4e7), (100.0, 1e5), (1000.0, 1e5)])
def test_masked_logits_under_large_entropy_gradients(dtype, scale, dh):
    """Masked logits have no gradient, whatever the scale and the entropy's gradient are."""
    x, t = masked(6, 9001, dtype, scale)
    r = run(x, t, scale, dh=dh)
    compare(x, t, scale, r)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("offset, scale", [(3000.0, 1.0), (-70000.0, 0.5), (50.0, 100.0)])
def test_masked_rows_far_from_zero(dtype, offset, scale):
    """|lse| of 1024 and more, where the backward takes differences to the largest logit, over several blocks a row."""
    x, t = masked(5, 20001, dtype, scale)
    x[x > -1e37] += offset
    r = run(x, t, scale, dh=1e9)
    assert bool((r["lse"].abs() >= 1024).all())
    compare(x, t, scale, r)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("scale", [0.5, 1.0, 2.0, 1000.0])
def test_finite_logits_whose_products_overflow(dtype, scale):
    """Rows of the type's lowest and largest values, alone and beside others: the probabilities depend on differences
    alone, in the forward and in its gradient; only what is itself past float32's range is infinite."""
    V, low, top = 1501, torch.finfo(DT[dtype]).min, torch.finfo(DT[dtype]).max
    x = torch.zeros(9, V)
    x[0] = low
    x[1], x[1, 40:] = -float("inf"), low     # equal ones, what is left of the row
    x[2], x[2, 700] = low, -1e37
    x[3] = top
    x[4], x[4, 1499] = low, top
    x[5, 3:900] = top
    x[6] = -2e38
    x[7] = -float("inf")
    x[8], x[8, 0] = -float("inf"), low
    x = x.to(DT[dtype]).cuda()
    t = torch.tensor([5, 50, 700, 1500, 1499, 3, 0, 1, 0], dtype=torch.int32, device="cuda")
    r = run(x, t, scale, K=7, dh=1.0)
    compare(x, t, scale, r, K=7)
    H = np.log([V, V - 40, 1, V, 1, 897, V, 1, 1])
    assert np.allclose(f64(r["entropy"]), H, atol=1e-4) and r["lse"][7].item() == -float("inf")


@pytest.mark.parametrize("scale", [0.7, 1.0, 3.0])
def test_large_finite_logits(scale):
    """Logits of any size between: equal ones are uniform, the next larger float is beside them or takes all."""
    size = torch.logspace(4, 38, 400, dtype=torch.float64).float()
    x = torch.cat([size, -size])[:, None].repeat(1, 601).cuda()
    x[::2, 77] = torch.nextafter(x[::2, 77], torch.full_like(x[::2, 77], float("inf")))
    t = torch.full((800,), 5, dtype=torch.int32, device="cuda")
    compare(x, t, scale, run(x, t, scale, K=3), K=3)


@pytest.mark.parametrize("N, V", [(2, 131072), (700, 16000)])
def test_overflowing_products_in_other_divisions_of_a_row(N, V):
    """The same in clusters of blocks and in narrow blocks."""
    for value in (torch.finfo(torch.float32).min, 3e38):
        x = torch.full((N, V), value, device="cuda")
        x[0, V // 2:] = -float("inf")
        t = torch.full((N,), V // 3, dtype=torch.int32, device="cuda")
        compare(x, t, 2.0, run(x, t, 2.0, K=3), K=3)


def test_no_entropy_without_its_gradient():
    """Without a gradient of the entropy the backward takes none, and an entropy that is given does not matter."""
    x, t = masked(5, 2003, "f32", 1.0)
    for offset in (0.0, 4000.0):
        x = x + offset
        want = run(x, t, 1.0)
        s = sdm.LogprobSpec(rows=5, V=2003, dtype="f32")
        outs = []
        for entropy in (None, want["entropy"], torch.full((5,), float("nan"), device="cuda")):
            outs.append(torch.full_like(x, float("nan")))
            sdm.token_logprobs_backward(s, x, t, want["lse"], entropy, want["d_logp"], outs[-1])
        d, e = logprobs_backward(f64(x), t.cpu().numpy(), 1.0, f64(want["d_logp"]), None)
        check("dlogits", outs[0], d, e)
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
        with pytest.raises(sdm.SdmError) as err:
            sdm.token_logprobs_backward(s, x, t, want["lse"], None, want["d_logp"], outs[0], d_entropy=want["d_entropy"])
        assert err.value.status == -1


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("pad", [0, 3])
def test_gradient_in_place_of_the_logits(dtype, pad):
    """Rows near zero and far from it (which every block of a row reads once more), empty ones among them."""
    N, V = 7, 50001
    buf = torch.zeros(N, V + pad, dtype=DT[dtype], device="cuda")
    x, t = masked(N, V, dtype, 1.0, seed=3)
    for i, offset in enumerate((0.0, 3000.0, -5000.0, 0.0, 1e6)):
        x[i][x[i] > -1e37] += offset
    x[5] = -float("inf")
    buf[:, :V] = x
    want = run(x, t, 1.0)
    compare(x, t, 1.0, want)
    s = sdm.LogprobSpec(rows=N, V=V, dtype=dtype)
    for _ in range(3):
        got = buf.clone()[:, :V]
        sdm.token_logprobs_backward(s, got, t, want["lse"], want["entropy"], want["d_logp"], got, want["d_entropy"])
        assert torch.equal(got, want["dlogits"])
