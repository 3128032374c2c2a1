"""The layer operators, the gradient set and the compressor in one training
loop: the example's gradients against automatic differentiation in 64 bits,
and its loss over the steps."""

import importlib.util
import os

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("train_block", os.path.join(ROOT, "examples", "train_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_gradients_of_the_whole_block(example):
    """Each of the five roundings between loss and weight (z, y and h, gate and
    up, dz, dy, dh, da and db) is half a step of bf16, 2^-8 at most of its
    element; they are independent, so the gradients' relative error in the
    2-norm stays under their sum, 8 * 2^-8."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    m, d, f, out = 130, 136, 328, 60
    block = example.Block(d, f, out, gen)
    p = example.Pass(block, m)
    x = torch.randn(m, d, generator=gen, device="cuda").to(torch.bfloat16)
    t = torch.randn(m, out, generator=gen, device="cuda").to(torch.bfloat16)
    z = p.forward(x)
    dz = ((z.float() - t.float()) / m).to(torch.bfloat16)
    got = dict(zip(block.weights, p.backward(x, dz)))
    w = {n: v.double().cpu().requires_grad_() for n, v in block.weights.items()}
    xd = x.double().cpu()
    h = torch.nn.functional.silu(xd @ w["wg"].t()) * (xd @ w["wu"].t())
    want_z = (xd + h @ w["wd"].t() + w["bd"]) @ w["wo"].t()
    assert float((z.double().cpu() - want_z.detach()).norm() / want_z.detach().norm()) < 4 * 2.0 ** -8
    want_z.backward(dz.double().cpu())
    for name, v in w.items():
        off = float((got[name].double().cpu() - v.grad).norm() / v.grad.norm())
        assert off < 8 * 2.0 ** -8, (name, off)


def test_the_loss_falls(example):
    losses = example.train(steps=40)
    assert losses[-1] < 0.5 * losses[0], losses[::8]
    assert losses == example.train(steps=40)
