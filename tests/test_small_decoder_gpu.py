"""The operators together, as the example uses them: its model learns streams that repeat, and answers them."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "small_decoder.py")


def example():
    spec = importlib.util.spec_from_file_location("small_decoder", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_the_model_learns_and_answers():
    ex = example()
    model = ex.SmallDecoder(P=2, C=48, S=128, hd=32, D=128, V=64)
    stream = ex.phrases(2, 64, 4 * 48 + 1, length=16)
    losses = model.train(stream, 15)
    assert losses[0] > 3.0 and losses[-1] < 0.5, losses   # log 64 = 4.16 before anything is learnt
    want = ex.phrases(2, 64, 4 * 48 + 17, length=16)[:, -16:]
    got = model.answer(stream[:, -1], 16)
    assert torch.equal(torch.stack([t for t, _, _ in got], 1), want)
    for t, vals, idx in got:
        assert torch.equal(idx[:, 0].long(), t) and bool((vals[:, :-1] >= vals[:, 1:]).all()) and bool((vals <= 0).all())


def test_the_losses_gradient_agrees_with_a_small_step():
    """A step of the output weights along their gradient lowers the loss by its square, to the curvature and bfloat16's
    rounding of the loss's inputs (a tenth)."""
    ex = example()
    model = ex.SmallDecoder(P=2, C=48, S=128, hd=32, D=128, V=64)
    s = ex.phrases(2, 64, 49, length=16)
    loss, d = model.train_chunk(s[:, :-1], s[:, 1:])
    for name in ("out", "x"):
        before = model.w[name].clone()
        eps = 0.02 / float(d[name].norm()) ** 2
        model.begin()
        model.w[name] = before - eps * d[name]
        lower, _ = model.train_chunk(s[:, :-1], s[:, 1:])
        model.begin()
        model.w[name] = before + eps * d[name]
        upper, _ = model.train_chunk(s[:, :-1], s[:, 1:])
        model.w[name] = before
        assert abs(float(upper - lower) / 0.04 - 1.0) < 0.1, name
