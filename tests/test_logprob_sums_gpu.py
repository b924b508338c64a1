"""The sums of the token log probabilities under bounds of their own depth, in every division of a row: a lost or doubled logit
does not fit them. The reference is the definition in torch float64.

Bounds (u = 2^-24). A row is read by `threads` threads, each of which takes its logits in batches of 16 or more, adds them in
pairs, moves its sums to a new reference at most once a batch, and joins with the others in at most 5 + 16 + 8 steps. With
t = (z - max z) / ln 2, E1 = sum p |t| and E2 = sum p t^2:
  * a term's way into the sum has one rounding for each addition, 6 for each move or join (2^t within 4 u, product, sum), 4 of
    its own 2^t; the exponents' roundings together 2 u |t|, since moves lead to the largest logit monotonically:
    the sum's relative error is rs = (D + 2 E1) u, D = additions + 6 (moves + joins) + 4;
  * the sum of 2^t t has terms of one sign: (D E1 + 3 E2) u;
  * scale log2(e) is rounded twice, and log2 and the last products are within 4 u each of what they give.
"""

import math

import numpy as np
import pytest
import torch

import sparse_slot_memory_gb300 as sdm

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24

# every division of a row: N, V, type, threads that read a row
FORMS = [(4, 131072, "bf16", 4096), (30, 131071, "bf16", 4096), (60, 70001, "bf16", 2048), (100, 40003, "f32", 1024),
         (10, 9001, "bf16", 1024), (1, 20011, "f32", 2048), (160, 60001, "f32", 256), (700, 30001, "bf16", 128),
         (1300, 5003, "bf16", 64), (200, 901, "f32", 64)]


def call(x, t, scale, K, d_logp=None, d_entropy=None):
    N, V = x.shape
    s = sdm.LogprobSpec(rows=N, V=V, K=K, dtype="bf16" if x.dtype == torch.bfloat16 else "f32", scale=scale)
    r = {k: torch.full((N,), float("nan"), device="cuda") for k in ("logp", "entropy", "lse")}
    r["top_vals"] = torch.full((N, K), float("nan"), device="cuda")
    r["top_idx"] = torch.full((N, K), -7, dtype=torch.int32, device="cuda")
    sdm.token_logprobs(s, x, t, r["logp"], r["entropy"], r["lse"], r["top_vals"], r["top_idx"])
    if d_logp is not None:
        r["dlogits"] = torch.full((N, V), float("nan"), dtype=x.dtype, device="cuda")
        sdm.token_logprobs_backward(s, x, t, r["lse"], r["entropy"], d_logp, r["dlogits"], d_entropy)
    return r


def within(name, got, want, tol):
    far = (got.double() - want).abs() - tol
    bad = ~(far <= 0) & ~(got.double() == want)   # equal infinities
    assert not bool(bad.any()), (name, int(bad.sum()), float(far.nan_to_num(1e30).max()), float(tol.max()))


def compare(x, t, scale, threads, r, d_logp=None, d_entropy=None):
    V, K = x.shape[1], r["top_idx"].shape[1]
    scale = float(np.float32(scale))
    z = x.double() * scale
    m = z.amax(1, keepdim=True)
    logs = torch.log_softmax(z, 1)
    lse = torch.logsumexp(z, 1)
    p = logs.exp()
    some = p > 0
    plogp = torch.where(some, p * logs, 0.0)
    H = -plogp.sum(1)
    d = torch.where(some, (z - m) / math.log(2), 0.0)
    E1, E2 = (p * d.abs()).sum(1), (p * d * d).sum(1)
    each = -(-V // threads)
    D = each / 2 + 16 + 31 + 6 * (each // 16 + 4 + 29) + 4
    rs = (D + 2 * E1) * U
    lg = math.log2(V) + 1
    lse_e = rs + U * (8 * (lse.abs() + m[:, 0].abs() + lg) + 4 * E1)
    H_e = 0.7 * (U * (D * E1 + 3 * E2) + rs * (E1 + 1.5)) + U * (8 * (lg + E1) + 2 * (E1 + E2))
    of = lambda v: rs[:, None] + U * (8 * v.abs().nan_to_num(posinf=0.0) + 8 * lg + 4 * E1[:, None])
    within("lse", r["lse"], lse, lse_e)
    within("entropy", r["entropy"], H, H_e)
    pick = logs.gather(1, t.long()[:, None])
    within("logp", r["logp"][:, None], pick, of(pick))
    # the lower id first among equals: a stable sort
    ids = torch.sort(x.float() + 0.0, dim=1, descending=True, stable=True).indices[:, :K]
    assert torch.equal(r["top_idx"].long(), ids)
    top = logs.gather(1, ids)
    within("top_vals", r["top_vals"], top, of(top))
    if d_logp is not None:
        one = torch.zeros_like(p).scatter_(1, t.long()[:, None], 1.0)
        dl, dh = d_logp.double()[:, None], d_entropy.double()[:, None]
        dz = dl * (one - p) - dh * (plogp + p * H[:, None])
        a = torch.where(some, logs, 0.0).abs()
        size = dl.abs() + dh.abs() * (a + H[:, None])
        tol = p * ((lse_e[:, None] + U * (6 * a + 14)) * size + dh.abs() * (lse_e + H_e)[:, None] + dh.abs() * 2 * U * a)
        tol = scale * (tol + 4 * U * (one * dl.abs() + dz.abs()))
        if x.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * (scale * dz.abs() + tol)
        within("dlogits", r["dlogits"], scale * dz, tol + 1e-37)
    return float(lse_e.max()), float(H_e.max())


def rows(N, V, dtype, scale, gen, pad=1):
    """Rows `pad` elements further apart than they are long, so that they lie differently on 16 bytes."""
    buf = torch.randn(N, V + pad, device="cuda", generator=gen) * scale
    return buf.to(DT[dtype])[:, :V]


@pytest.mark.parametrize("N, V, dtype, threads", FORMS)
@pytest.mark.parametrize("masked", [False, True])
def test_random_rows(N, V, dtype, threads, masked):
    gen = torch.Generator(device="cuda").manual_seed(V + masked)
    x = rows(N, V, dtype, 3.0, gen)
    if masked:
        u = torch.rand(V, device="cuda", generator=gen)
        x[:, u < 0.2] = -float("inf")
        x[:, (u > 0.5) & (u < 0.7)] = torch.finfo(DT[dtype]).min
    t = torch.randint(0, V, (N,), device="cuda", generator=gen, dtype=torch.int32)
    dl, dh = (torch.randn(N, device="cuda", generator=gen) for _ in range(2))
    lse_e, _ = compare(x, t, 0.7, threads, call(x, t, 0.7, 20, dl, dh), dl, dh)
    assert lse_e < 1.2e-4   # a fraction of a logit's share of the sum, not of the whole row's


def places(V, per):
    """Ids at the ends of a row, of the parts of 2, 4 and 8 blocks and of batches, and a few between."""
    near = lambda i: range(i - 9, i + 10)
    ids = set(range(20)) | set(range(V - 20, V))
    for parts in (2, 4, 8):
        for k in range(1, parts):
            ids |= set(near(k * V // parts)) | set(near(k * (-(-(V // per) // parts)) * per))
    for step in (1024, 2048, 4096, 8192, 16384):
        ids |= set(near(V // step * step))
    ids |= set(np.random.default_rng(V).integers(0, V, 40).tolist())
    return sorted(i for i in ids if 0 <= i < V)


@pytest.mark.parametrize("N, V, dtype, threads", FORMS)
def test_one_logit_holds_the_row(N, V, dtype, threads):
    """All of a row's mass on one logit, at every place where a division of the row begins or ends: left out, lse moves by
    about 20; counted twice, by ln 2."""
    gen = torch.Generator(device="cuda").manual_seed(V)
    ids = torch.tensor(places(V, 8 if dtype == "bf16" else 4), device="cuda")
    for i in range(0, len(ids), N):
        at = ids[i:i + N]
        at = torch.cat([at, ids[:N - len(at)]]) if len(at) < N else at
        at = at.repeat(-(-N // len(at)))[:N]
        x = rows(N, V, dtype, 1.0, gen, pad=3)
        x[torch.arange(N, device="cuda"), at] = 36.0
        t = at.to(torch.int32)
        dl, dh = (torch.randn(N, device="cuda", generator=gen) for _ in range(2))
        compare(x, t, 1.0, threads, call(x, t, 1.0, 3, dl, dh), dl, dh)


@pytest.mark.parametrize("N, V, dtype, threads", FORMS)
def test_rows_with_nan_or_little_left(N, V, dtype, threads):
    """NaN and +inf in their rows, rows with nothing left, one logit left, and equal lowest values, in every division."""
    gen = torch.Generator(device="cuda").manual_seed(V + 7)
    for seed in range(max(1, 8 // N)):
        x = rows(N, V, dtype, 2.0, gen)
        t = torch.randint(0, V, (N,), device="cuda", generator=gen, dtype=torch.int32)
        kind = (torch.arange(N, device="cuda") + seed * N) % 8
        at = torch.randint(0, V, (N,), device="cuda", generator=gen)
        low = torch.finfo(DT[dtype]).min
        for n in range(N):
            k, i = int(kind[n]), int(at[n])
            if k in (1, 2):
                x[n, i] = (float("nan"), float("inf"))[k - 1]
            elif k in (3, 4):
                x[n] = -float("inf")
                if k == 4:
                    x[n, i] = -3.0
                    t[n] = i
            elif k == 5:
                x[n] = low
            elif k == 6:
                x[n], x[n, i] = low, -5.0
        dl, dh = (torch.randn(N, device="cuda", generator=gen) for _ in range(2))
        r = call(x, t, 1.0, 5, dl, dh)
        bad, none, wide = (kind == 1) | (kind == 2), kind == 3, kind == 5
        for k in ("lse", "logp", "entropy", "top_vals", "dlogits"):
            assert bool(r[k][bad].isnan().all()), k
        assert torch.equal(r["top_idx"][bad][:, 0].long(), at[bad])
        assert bool((r["lse"][none] == -float("inf")).all()) and bool((r["entropy"][none] == 0).all())
        assert bool((r["logp"][none] == -float("inf")).all())
        assert r["top_idx"][none].tolist() == [list(range(5))] * int(none.sum())
        one = torch.zeros(N, V, device="cuda").scatter_(1, t.long()[:, None], 1.0)
        assert torch.equal(r["dlogits"][none], (dl[:, None] * one).to(x.dtype)[none])
        # equal lowest values: differences to the largest are exact, the sum is V
        H = torch.full((N,), math.log(V), device="cuda", dtype=torch.float64)
        within("uniform entropy", r["entropy"][wide], H[wide], 16 * U * H[wide])
        within("uniform logp", r["logp"][wide], -H[wide], 16 * U * H[wide])
        g = dl[:, None].double() * (one - 1.0 / V)   # the entropy is at its largest: no gradient of it
        tol = 64 * U * (dl.abs() + dh.abs() * math.log(V))[:, None].double() / V + 4 * U * g.abs()
        tol = tol + (2.0 ** -8 * g.abs() if dtype == "bf16" else 0.0)
        within("uniform gradient", r["dlogits"][wide], g[wide], tol[wide])
        fine = ~(bad | none | wide)
        if bool(fine.any()):
            part = {k: v[fine] for k, v in r.items()}
            compare(x[fine], t[fine], 1.0, threads, part, dl[fine], dh[fine])
