"""The token operators together with the layers, the gradient set and the
compressor in one training loop: the example's gradients against automatic
differentiation in 64 bits, its steps one token at a time against the whole
texts, and that it runs."""

import importlib.util
import math
import os

import pytest
import torch

import token_reference as R
from conftest import ROOT

pytestmark = pytest.mark.gpu
F = torch.nn.functional


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("train_tokens", os.path.join(ROOT, "examples", "train_tokens.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def logits(w, ids, batch, scale, p, seed, use):
    """The model's formula in 64 bits on the CPU."""
    d, m = w["table"].shape[1], len(ids)

    def drop(x, offset):
        kept = R.kept(p)
        return torch.where(torch.from_numpy(R.draws(m, d, seed, offset) < kept), x * (65536 / kept), 0.0)

    def norm(x, name):
        return F.layer_norm(x, (d,), w[name + "w"], w[name + "b"], 1e-5)

    x = drop(w["table"][ids] * scale, 2 * use)
    gx = norm(x, "n1") @ w["wi"].t() + w["bi"]
    f, u = torch.sigmoid(gx[:, :d]).view(batch, -1, d), (torch.sigmoid(-gx[:, :d]) * gx[:, d:]).view(batch, -1, d)
    now, rows = torch.zeros(batch, d, dtype=torch.float64), []
    for t in range(f.shape[1]):
        now = f[:, t] * now + u[:, t]
        rows.append(now)
    y1 = x + torch.stack(rows, 1).reshape(m, d) @ w["wo"].t()
    c = norm(y1, "n2")
    y2 = y1 + drop((F.silu(c @ w["wg"].t()) * (c @ w["wu"].t())) @ w["wd"].t(), 2 * use + 1)
    return norm(y2, "n3") @ w["table"].t()


def test_gradients_of_the_whole_model(example):
    """Some 20 tensors between the loss and a weight are rounded to bf16, by 2^-8 of an element at most and
    independently, so the gradients' relative error in the 2-norm stays under their sum, 20 * 2^-8; the logits',
    behind ten of them, under 10 * 2^-8."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    batch, length, vocab, use = 5, 37, 61, 4
    model = example.Model(vocab, 104, 152, gen)
    for name in ("n1b", "n2b", "n3b", "bi"):
        model.weights[name].copy_(0.3 * torch.randn(model.weights[name].shape, generator=gen, device="cuda"))
    run = example.Pass(model, batch, length, 0.25)
    ids = torch.randint(0, vocab, (batch * length,), generator=gen, device="cuda")
    dz = (torch.randn(len(ids), vocab, generator=gen, device="cuda") / len(ids)).to(torch.bfloat16)
    z = run.forward(ids, use).double().cpu()
    got = dict(zip(model.weights, run.backward(ids, use, dz)))
    w = {n: v.double().cpu().requires_grad_() for n, v in model.weights.items()}
    want = logits(w, ids.cpu(), batch, model.scale, run.p, example.SEED, use)
    assert float((z - want.detach()).norm() / want.detach().norm()) < 10 * 2.0 ** -8
    want.backward(dz.double().cpu())
    for name, v in w.items():
        off = float((got[name].double().cpu() - v.grad).norm() / v.grad.norm())
        assert off < 20 * 2.0 ** -8, (name, off)


def test_token_by_token_is_the_whole_text(example):
    """The same logits, up to roundings, from one token of each text at a time with the states handed on."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    batch, length, vocab = 6, 9, 50
    model = example.Model(vocab, 72, 136, gen)
    ids = torch.randint(0, vocab, (batch, length), generator=gen, device="cuda")
    whole = example.Pass(model, batch, length, 0.0)
    want = whole.forward(ids.reshape(-1), 0).clone().view(batch, length, vocab).float()
    step = example.Pass(model, batch, 1, 0.0)
    state = torch.zeros(batch, 72, device="cuda")
    for t in range(length):
        z = step.forward(ids[:, t].contiguous(), 0, h0=state).float()
        state.copy_(step.state)
        assert float((z - want[:, t]).norm() / want[:, t].norm()) < 10 * 2.0 ** -8, t
    # the state in 32 bits, behind a product of other shape in bf16
    assert float((state - whole.state).norm() / whole.state.norm()) < 4 * 2.0 ** -8


def test_it_runs_and_gives_the_same_twice(example):
    losses = example.train(steps=6)
    assert all(math.isfinite(v) for v in losses) and losses == example.train(steps=6)
