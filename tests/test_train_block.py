"""The example's training step: layer, norm, gradient norm and optimizer together."""
import importlib.util
import os

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("train_block", os.path.join(ROOT, "examples", "train_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("bits", [8, 32])
def test_the_loss_falls(example, bits):
    losses = example.train(steps=48, bits=bits)
    first, last = sum(losses[:4]) / 4, sum(losses[-4:]) / 4
    assert all(x == x and x < 10 * first for x in losses)
    assert last < 0.6 * first, (first, last)


def test_a_run_repeats_its_losses(example):
    assert example.train(steps=8, log=lambda *a: None) == example.train(steps=8, log=lambda *a: None)


def test_gradients_against_differences(example):
    """The block's gradient along a random direction against the loss's slope there, from fp64 sums of
    bf16 outputs.  Each output is off by 2^-8 of itself at most, at random: over 2 * 100352 outputs
    that moves the difference quotient by well under a tenth of the slope at this step."""
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(5)
    block = example.Block(2, 64, 28, 28, 8, "gelu", dev)
    masters = block.init(gen)
    x = torch.randn((2, 64, 28, 28), generator=gen, device=dev).bfloat16()
    dy = torch.randn(x.shape, generator=gen, device=dev).bfloat16()
    # gamma and beta stay exact in bf16 along the way, so the quotient is theirs alone
    params = {k: v.bfloat16() for k, v in masters.items()}
    grads = {k: torch.zeros_like(v) for k, v in params.items()}
    _, saved = block.forward(x, params)
    block.backward(x, params, saved, dy, grads)

    def loss(p):
        return (block.forward(x, p)[0].double() * dy.double()).sum()

    for name in ("gamma", "beta"):
        direction = torch.sign(grads[name].float())
        moved = {s: dict(params) for s in (1, -1)}
        for s in (1, -1):
            moved[s][name] = (params[name].float() + s * 0.0625 * direction).bfloat16()
        way = (moved[1][name].double() - moved[-1][name].double())
        slope = (grads[name].double() * way).sum()
        assert abs((loss(moved[1]) - loss(moved[-1])) / slope - 1) < 0.1
