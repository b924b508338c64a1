"""The small decoder's gradients, written by hand around the operators, against the same model in 64 bits, differentiated by torch:
of a chunk that follows another, with states of the recurrence and of the delta rule, positions, and an empty memory.

The example computes in bfloat16 rows. The same 64-bit model with every row, weight and row's gradient rounded to bfloat16 is off by
`rounded`, of each weight's gradient in the root of its squares; the example rounds in the same places, so 3 times that is allowed."""

import pytest
import torch
import torch.nn.functional as F

from test_small_decoder_gpu import example

NAMES = ("emb", "x", "g", "qkv", "gb", "n1", "n2", "n3", "n4", "out")


class Round(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x):
        return x.bfloat16().double()

    @staticmethod
    def backward(ctx, d):
        return d.bfloat16().double()


def norm(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


PATHS = ("gates", "inputs", "stream", "rule", "rule's gates", "second stream", "lengths")


def loss_of(w, tokens, targets, h0, s0, hd, rnd, cut=None):
    """The mean loss of a chunk [P, C] from the states h0 [P, D], s0 [P, H, hd, hd], and the states after. No gradient passes `cut`."""
    past = lambda name, t: t.detach() if name == cut else t
    P, C = tokens.shape
    D = w["emb"].shape[1]
    H = D // hd
    b = {n: rnd(t) if t.dim() == 2 and n != "emb" else t for n, t in w.items()}   # products take bfloat16 weights
    e = rnd(w["emb"][tokens])
    g = F.logsigmoid(rnd(past("gates", e) @ b["g"]) + 2.0)
    x = rnd(past("inputs", e) @ b["x"])
    h, hs = h0, []
    for t in range(C):
        h = g[:, t].exp() * h + x[:, t]
        hs.append(h)
    r1 = rnd(past("stream", e) + norm(rnd(torch.stack(hs, 1))) * w["n1"])
    y1 = rnd(norm(r1) * w["n2"])
    q, k, v = rnd(past("rule", y1) @ b["qkv"]).view(P, C, 3, H, hd).unbind(2)
    unit = lambda t: rnd(t * torch.rsqrt(past("lengths", t).square().sum(-1, keepdim=True) + 1e-6))
    q, k = unit(q), unit(k)
    a, beta = rnd(past("rule's gates", y1) @ b["gb"]).split((H, H), 2)
    a, beta = torch.sigmoid(a + 3.0), torch.sigmoid(beta)
    S, us = s0, []
    for t in range(C):
        S = S * a[:, t, :, None, None]
        S = S + k[:, t, :, :, None] * (beta[:, t, :, None] * (v[:, t] - (S * k[:, t, :, :, None]).sum(2)))[:, :, None, :]
        us.append((S * q[:, t, :, :, None]).sum(2) * hd ** -0.5)
    r2 = rnd(past("second stream", r1) + norm(rnd(torch.stack(us, 1)).view(P, C, D)) * w["n3"])
    logits = rnd(rnd(norm(r2) * w["n4"]) @ b["out"])
    return F.cross_entropy(logits.view(P * C, -1), targets.reshape(-1)), h, S


def gradients(w, tokens, targets, h0, s0, hd, rnd=lambda t: t, cut=None):
    leaf = {n: w[n].detach().double().cpu().requires_grad_() for n in NAMES}
    loss, h, s = loss_of(leaf, tokens, targets, h0, s0, hd, rnd, cut)
    loss.backward()
    return float(loss.detach()), {n: t.grad for n, t in leaf.items()}, h.detach(), s.detach()


def off(got, want):
    return {n: float((got[n] - want[n]).norm() / want[n].norm()) for n in NAMES}


@pytest.mark.gpu
def test_gradients_of_a_second_chunk():
    ex = example()
    P, C, hd = 2, 48, 32
    model = ex.SmallDecoder(P=P, C=C, S=128, hd=hd, D=128, V=64)
    gen = torch.Generator(device="cuda").manual_seed(5)
    for n in ("n1", "n2", "n3", "n4"):
        model.w[n].add_(torch.randn(128, device="cuda", generator=gen), alpha=0.2)
    s = ex.phrases(P, 64, 2 * C + 1, length=16)
    model.train_chunk(s[:, :C], s[:, 1:C + 1])
    model.bank.zero_()
    h0, s0 = model.h.double().cpu(), model.s.double().cpu()
    loss, d = model.train_chunk(s[:, C:2 * C], s[:, C + 1:])
    got = {n: d[n].double().cpu() for n in NAMES}
    tokens, targets = s[:, C:2 * C].cpu(), s[:, C + 1:].cpu()
    value, want, h, S = gradients(model.w, tokens, targets, h0, s0, hd)
    near, rounded, _, _ = gradients(model.w, tokens, targets, h0, s0, hd, Round.apply)
    assert abs(float(loss) - value) <= 3 * abs(near - value) + 1e-2
    lim, is_ = off(rounded, want), off(got, want)
    for n in NAMES:
        assert is_[n] <= 3 * lim[n] + 2.0 ** -9, (n, is_[n], lim[n])
    assert float((model.h.double().cpu() - h).norm() / h.norm()) <= 2.0 ** -7
    assert float((model.s.double().cpu() - S).norm() / S.norm()) <= 2.0 ** -6


def test_a_path_that_is_left_out_would_show():
    """Each path that the gradients take makes more of a difference than is allowed, in a model of the same sizes on the CPU."""
    P, C, hd, D, V = 2, 48, 32, 128, 64
    gen = torch.Generator().manual_seed(0)
    rand = lambda *n: torch.randn(*n, generator=gen)
    w = {"emb": rand(V, D), "out": rand(D, V) * D ** -0.5} | {n: 1 + 0.2 * rand(D) for n in ("n1", "n2", "n3", "n4")}
    w |= {n: rand(D, m) * D ** -0.5 for n, m in (("x", D), ("g", D), ("qkv", 3 * D), ("gb", 2 * D // hd))}
    tokens = torch.randint(V, (P, 16), generator=gen).repeat(1, 4)[:, :C + 1]
    args = (w, tokens[:, :-1], tokens[:, 1:], rand(P, D).double(), 0.3 * rand(P, D // hd, hd, hd).double(), hd)
    _, want, _, _ = gradients(*args)
    lim = off(gradients(*args, Round.apply)[1], want)
    for cut in PATHS:
        without = off(gradients(*args, cut=cut)[1], want)
        assert any(without[n] > 2 * (3 * lim[n] + 2.0 ** -9) for n in NAMES), cut
