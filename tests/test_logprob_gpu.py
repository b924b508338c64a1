"""Log probabilities of given tokens with entropy and top alternatives, and the logits' gradient
(sdm_token_logprobs, sdm_token_logprobs_backward), against their definition in 64 bits (tests/operators_testlib.py, which
derives the bounds). Ids are compared exactly."""

import numpy as np
import pytest
import torch

import sparse_slot_memory_gb300 as sdm
from operators_testlib import check, f64, logprobs, logprobs_backward, order_topk
from sparse_slot_memory_gb300 import _abi

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def run(x, targets, K, scale=1.0, d_entropy=True, seed=9):
    """Forward and backward of logits x (a CUDA tensor [N, V], rows any distance apart)."""
    N, V = x.shape
    name = "bf16" if x.dtype == torch.bfloat16 else "f32"
    s = sdm.LogprobSpec(rows=N, V=V, K=K, dtype=name, scale=scale)
    gen = torch.Generator().manual_seed(seed)
    r = {k: torch.full((N,), float("nan"), device="cuda") for k in ("logp", "entropy", "lse")}
    r["top_vals"] = torch.full((N, K), float("nan"), device="cuda")
    r["top_idx"] = torch.full((N, K), -7, dtype=torch.int32, device="cuda")
    r["d_logp"] = torch.randn(N, generator=gen).cuda()
    r["d_entropy"] = torch.randn(N, generator=gen).cuda() if d_entropy else None
    r["dlogits"] = torch.full((N, V), float("nan"), dtype=x.dtype, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sdm.token_logprobs(s, x, targets, r["logp"], r["entropy"], r["lse"], r["top_vals"], r["top_idx"], status=st)
    sdm.token_logprobs_backward(s, x, targets, r["lse"], r["entropy"], r["d_logp"], r["dlogits"], r["d_entropy"], status=st)
    r["status"] = int(st.item())
    return r


def compare(x, targets, K, scale, r):
    X, t = f64(x), targets.cpu().numpy()
    scale = float(np.float32(scale))
    f = logprobs(X, t, scale)
    check("logp", r["logp"], f["logp"], f["logp_e"])
    check("entropy", r["entropy"], f["H"], f["H_e"])
    check("lse", r["lse"], f["lse"], f["lse_e"])
    if K:
        top = order_topk(X, K)
        assert np.array_equal(r["top_idx"].cpu().numpy(), top)
        at = (np.arange(len(X))[:, None], top)
        check("top_vals", r["top_vals"], f["logs"][at], f["logs_e"][at])
    d, e = logprobs_backward(X, t, scale, f64(r["d_logp"]), None if r["d_entropy"] is None else f64(r["d_entropy"]))
    check("dlogits", r["dlogits"], d, e, x.dtype)


def logits(N, V, dtype, pad=0, seed=0, scale=3.0):
    gen = torch.Generator().manual_seed(seed)
    t = torch.full((N, V + pad), float("nan"))
    t[:, :V] = torch.randn(N, V, generator=gen) * scale
    return t.to(DT[dtype]).cuda()[:, :V]


def targets(N, V, seed=1):
    t = torch.randint(0, V, (N,), generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    if N > 2:
        t[1], t[2] = -100, V - 1
    return t.cuda()


@pytest.mark.parametrize("N, V, K, dtype, pad, scale", [
    (1, 1, 1, "f32", 0, 1.0), (1, 1, 0, "bf16", 0, 1.0), (3, 2, 2, "bf16", 0, 1.0), (4, 7, 7, "f32", 0, 0.5),
    (5, 31, 31, "bf16", 0, 1.0), (5, 33, 32, "bf16", 2, 1.0), (3, 255, 5, "f32", 1, 2.0), (7, 1000, 20, "bf16", 0, 1.0),
    (9, 1001, 20, "bf16", 0, 0.7), (3, 4099, 32, "f32", 3, 1.0), (2, 8193, 1, "bf16", 5, 1.0),
    (1, 32003, 20, "bf16", 0, 1.3), (2, 50001, 10, "f32", 0, 1.0), (200, 513, 8, "bf16", 0, 1.0),
    (1, 131072, 20, "bf16", 0, 1.0)])
def test_forward_and_backward(N, V, K, dtype, pad, scale):
    x, t = logits(N, V, dtype, pad), targets(N, V)
    r = run(x, t, K, scale)
    assert r["status"] == 0
    compare(x, t, K, scale, r)


def test_masked_logits_and_rows_with_nothing_left():
    """-inf, the type's lowest value, whole rows of either (nothing left; equal logits), one logit left."""
    for dtype in ("f32", "bf16"):
        x, t = logits(8, 1003, dtype), targets(8, 1003)
        low = torch.finfo(DT[dtype]).min
        x[0, ::2] = -float("inf")
        x[1, 1::3] = low
        x[2] = -float("inf")
        x[3] = low
        x[4] = -float("inf")
        x[4, 700] = 2.0
        x[5, :] = -1e32
        x[6, 5:] = -float("inf")
        x[6, 5] = low
        t[0], t[4] = 2, 700
        r = run(x, t, 10)
        compare(x, t, 10, 1.0, r)
        assert r["lse"][2].item() == -float("inf") and r["entropy"][2].item() == 0
        assert r["top_idx"][2].tolist() == list(range(10)) and r["top_idx"][3].tolist() == list(range(10))


def test_equal_logits_go_to_the_lowest_id():
    x, t = torch.zeros(4, 5000, device="cuda"), targets(4, 5000)
    x[1] = (torch.arange(5000, device="cuda") % 7).float()
    x[2, 4000:] = 1.0
    x[3] = -torch.zeros(5000, device="cuda")
    x[3, 17] = 0.0
    for dt in DT.values():
        compare(x.to(dt), t, 32, 1.0, run(x.to(dt), t, 32))


def test_ascending_and_descending_rows():
    x = torch.arange(20000, device="cuda", dtype=torch.float32)[None] * 1e-3
    x = torch.cat([x, x.flip(1), x.roll(77, 1)])
    t = targets(3, 20000)
    compare(x, t, 20, 1.0, run(x, t, 20))


def test_large_offsets():
    """Logits far from 0: probabilities depend on differences alone, and keep their precision."""
    x, t = logits(4, 3001, "f32", scale=1.0).round(decimals=1), targets(4, 3001)
    x += torch.tensor([3000.0, -50000.0, 1e6, 20.0], device="cuda")[:, None]
    compare(x, t, 5, 1.0, run(x, t, 5))


def test_nan_and_infinity_stay_in_their_row():
    x, t = logits(6, 2000, "f32"), targets(6, 2000)
    clean = run(x, t, 5)
    x[1, 77], x[3, 0], x[3, 1999] = float("nan"), float("inf"), -float("inf")
    r = run(x, t, 5)
    ok = [0, 2, 4, 5]
    for k in ("logp", "entropy", "lse", "top_vals", "top_idx", "dlogits"):
        assert torch.equal(r[k][ok], clean[k][ok]), k
    assert bool(torch.isnan(r["lse"][[1, 3]]).all()) and bool(torch.isnan(r["entropy"][[1, 3]]).all())
    assert bool(torch.isnan(r["top_vals"][[1, 3]]).all())
    assert r["top_idx"][1, 0].item() == 77 and r["top_idx"][3, 0].item() == 0


def test_bad_targets_are_ignored_and_reported():
    x = logits(4, 100, "f32")
    t = torch.tensor([5, 100, -1, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    r = run(x, t, 3)
    assert r["status"] == _abi.SDM_DEV_BAD_TARGET
    assert r["logp"][1:].tolist() == [0, 0, 0]
    compare(x, t, 3, 1.0, r)


def test_optional_outputs_and_repeated_calls():
    x, t = logits(5, 3000, "bf16"), targets(5, 3000)
    a, b = run(x, t, 7), run(x, t, 7)
    for k in ("logp", "entropy", "lse", "top_vals", "top_idx", "dlogits"):
        assert torch.equal(a[k], b[k]), k
    s = sdm.LogprobSpec(rows=5, V=3000, K=7)
    logp, idx = torch.empty(5, device="cuda"), torch.empty(5, 7, dtype=torch.int32, device="cuda")
    sdm.token_logprobs(s, x, t, logp)
    assert torch.equal(logp, a["logp"])
    sdm.token_logprobs(s, x, t, logp, top_idx=idx)
    assert torch.equal(idx, a["top_idx"])
    r = run(x, t, 7, d_entropy=False)
    compare(x, t, 7, 1.0, r)


def test_gradient_agrees_with_differences():
    """Against central differences of the 64-bit definition along random directions (step 1e-4: a relative error below
    1e-6), the float32 gradient's own error and no other."""
    x, t = logits(6, 501, "f32", scale=2.0), targets(6, 501)
    for scale in (1.0, 0.6):
        r = run(x, t, 0, scale)
        X, tt = f64(x), t.cpu().numpy()
        sc = float(np.float32(scale))

        def loss(v):
            f = logprobs(v, tt, sc)
            return (f["logp"] * f64(r["d_logp"])).sum() + (f["H"] * f64(r["d_entropy"])).sum()

        v = np.random.default_rng(4).standard_normal(X.shape)
        want = (loss(X + 1e-4 * v) - loss(X - 1e-4 * v)) / 2e-4
        terms = f64(r["dlogits"]) * v
        assert abs(terms.sum() - want) <= 1e-5 * np.abs(terms).sum()


def test_rows_past_32_bits():
    """More than 2^31 logits: the last rows lie behind them."""
    N, V = 34000, 65001
    x = torch.empty(N, V, dtype=torch.bfloat16, device="cuda").normal_().mul_(2)
    t = targets(N, V)
    r = run(x, t, 3)
    at = [0, N // 2, N - 2, N - 1]
    part = {k: v[at] if isinstance(v, torch.Tensor) else v for k, v in r.items()}
    compare(x[at], t[at], 3, 1.0, part)


def test_rows_of_the_gradient_that_lie_differently():
    """The gradient's rows on another 16-byte offset than the logits'."""
    x, t = logits(5, 1001, "bf16", pad=7), targets(5, 1001)
    want = run(x, t, 0)
    s = sdm.LogprobSpec(rows=5, V=1001)
    buf = torch.zeros(5, 1003, dtype=torch.bfloat16, device="cuda")
    sdm.token_logprobs_backward(s, x, t, want["lse"], want["entropy"], want["d_logp"], buf[:, 1:1002], want["d_entropy"])
    assert torch.equal(buf[:, 1:1002], want["dlogits"]) and bool((buf[:, [0, 1002]] == 0).all())


def test_no_rows_and_refusals():
    s = sdm.LogprobSpec(rows=0, V=100, K=3, dtype="f32")
    e = torch.empty(0, device="cuda")
    sdm.token_logprobs(s, torch.empty(0, 100, device="cuda"), e.int(), e, e, e, e.view(0, 3), e.int().view(0, 3))
    x, t, o = logits(4, 100, "f32"), targets(4, 100), torch.empty(4, device="cuda")
    s = sdm.LogprobSpec(rows=4, V=100, K=3, dtype="f32")
    with pytest.raises(ValueError, match="logits: expected shape"):
        sdm.token_logprobs(s, x[:, :99], t, o)
    with pytest.raises(TypeError, match="targets"):
        sdm.token_logprobs(s, x, t.long(), o)
    with pytest.raises(ValueError, match="top_idx"):
        sdm.token_logprobs(s, x, t, o, top_idx=torch.empty(4, 2, dtype=torch.int32, device="cuda"))
    for bad in (dict(K=33), dict(K=101, V=100), dict(scale=0.0), dict(scale=float("nan")), dict(V=0, K=0)):
        b = sdm.LogprobSpec(**{**dict(rows=4, V=100, K=3, dtype="f32"), **bad})
        assert _abi.load().sdm_token_logprobs(b.c(), x.data_ptr(), 100, t.data_ptr(), o.data_ptr(), None, None, None, None,
                                              None, None) == -2, bad


@pytest.mark.parametrize("N, V, K, dtype", [
    (1300, 5003, 20, "bf16"), (1216, 2999, 32, "f32"), (1217, 12289, 1, "bf16"), (620, 14001, 20, "bf16"),
    (608, 3501, 32, "f32"), (760, 33000, 7, "bf16"), (607, 7001, 17, "bf16")])
def test_many_rows_take_narrow_blocks(N, V, K, dtype):
    """The block widths that many rows get, with ties, masked logits and rows with nothing left among them."""
    x, t = logits(N, V, dtype, pad=1), targets(N, V)
    x[3] = -float("inf")
    x[4] = 1.0
    x[5, ::2] = torch.finfo(DT[dtype]).min
    x[6] = torch.arange(V, device="cuda") * 1e-3
    x[7, : V - 1] = -float("inf")
    x[N - 1] = torch.arange(V, device="cuda").flip(0) * 1e-3
    compare(x, t, K, 1.0, run(x, t, K))


@pytest.mark.parametrize("N, V, dtype", [(2, 131072, "bf16"), (3, 70001, "f32"), (40, 30000, "bf16"), (620, 4500, "bf16")])
@pytest.mark.parametrize("K", [1, 20, 32])
def test_ties_across_the_threads_of_a_row(N, V, dtype, K):
    """Few different values, so that the K-th largest has equals in every part of a row; the lowest ids have to win."""
    x, t = logits(N, V, dtype, scale=1.0).float().round(), targets(N, V)
    x[0] = x[0].clamp(max=2.0)
    x[1] = x[1].clamp(max=2.0)
    x[1, V - 9:] = 3.0
    x[1, 5] = 3.0
    x = x.to(DT[dtype])
    compare(x, t, K, 1.0, run(x, t, K))
