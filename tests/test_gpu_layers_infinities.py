"""Infinite values in the operands of the layer gradients: each output is
infinite, NaN or finite where its formula in 64 bits is, whatever the number
of rows (up to 32 of them dz is kept in two halves, and a half that is 0 or of
the other sign would make NaN of an infinity)."""

import pytest
import torch

import layer_reference as R
from gpu_harness import say
from sparsified_gradient_compression_amd import dgc

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dgc.lib()
    return torch


def normal(seed, *shape):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda")


def same_kind(name, got, want):
    """NaN, infinite of either sign, or finite, element by element."""
    got = got.cpu()
    for what, g, w in (("nan", torch.isnan(got), torch.isnan(want)), ("+inf", got == INF, want == INF),
                       ("-inf", got == -INF, want == -INF)):
        assert torch.equal(g, w), (name, what, int((g != w).sum()), (g != w).nonzero()[0].tolist())


def host(*tensors):
    return [t.double().cpu() for t in tensors]


def product(a, b):
    """a b term by term: a matrix product may leave out terms that are 0 times something."""
    return (a[:, :, None] * b[None]).sum(1)


@pytest.mark.parametrize("m", (1, 7, 32, 33, 130))
@pytest.mark.parametrize("act", ("relu", "silu", "gelu"))
@pytest.mark.parametrize("dtype", (BF16, FP16))
@pytest.mark.parametrize("n,k", [(64, 72), (200, 35)])
def test_infinite_operands_of_linear_backward(m, n, k, dtype, act):
    say(f"infinities {m} {n} {k} {dtype} {act}")
    dy, x, pre = normal(1, m, n).to(dtype), normal(2, m, k).to(dtype), normal(3, m, n).to(dtype)
    w = (normal(4, n, k) * k ** -0.5).to(dtype)
    dy[0, 5] = 1.5  # exact in 16 bits: behind relu with a slope of 1 nothing is lost in rounding
    pre[0] = pre[0].abs() + 0.25
    w[5, 3], w[9, 4] = INF, -INF
    x[0, 2], x[m - 1, 8] = INF, -INF
    dx, dw = torch.empty_like(x), torch.empty(n, k, device="cuda")
    dgc.linear_backward(dy, x, w, pre, act, dx, dw)
    dyd, xd, wd, pred = host(dy, x, w, pre)
    dz = dyd * R.act_pair(act, pred)[1]
    same_kind("dx", dx, product(dz, wd))
    same_kind("dw", dw, product(dz.t(), xd))


@pytest.mark.parametrize("m", (1, 7, 32, 33, 130))
@pytest.mark.parametrize("act", ("relu", "silu"))
@pytest.mark.parametrize("dtype", (BF16, FP16))
def test_infinite_operands_of_gated_ffn_backward(m, dtype, act):
    d, f = 72, 136
    say(f"gated infinities {m} {dtype} {act}")
    dh, x = normal(1, m, f).to(dtype), normal(2, m, d).to(dtype)
    gate, up = normal(3, m, f).to(dtype), normal(4, m, f).to(dtype)
    wg, wu = ((normal(s, f, d) * d ** -0.5).to(dtype) for s in (5, 6))
    gate[0] = gate[0].abs() + 0.25
    dh[0, 5], up[0, 5] = 1.5, 2.0
    wg[5, 3], wu[9, 4], x[0, 2], x[m - 1, 8] = INF, -INF, INF, -INF
    dx, dg, du = torch.empty_like(x), torch.empty(f, d, device="cuda"), torch.empty(f, d, device="cuda")
    dgc.gated_ffn_backward(dh, x, wg, wu, gate, up, act=act, dx=dx, dw_gate=dg, dw_up=du)
    h, xd, a, b, g64, u64 = host(dh, x, gate, up, wg, wu)
    value, slope = R.act_pair(act, a)
    da, db = h * b * slope, h * value
    same_kind("dx", dx, product(da, g64) + product(db, u64))
    same_kind("dw_gate", dg, product(da.t(), xd))
    same_kind("dw_up", du, product(db.t(), xd))


@pytest.mark.parametrize("dtype", (BF16, FP16))
@pytest.mark.parametrize("m", (2, 40))
def test_infinite_and_nan_gradients(m, dtype):
    """An infinite dz is one in both halves, and a NaN too."""
    n, k = 64, 48
    dy, x, pre = normal(1, m, n).to(dtype), normal(2, m, k).to(dtype), normal(3, m, n).to(dtype)
    w = normal(4, n, k).to(dtype)
    dy[0, 7], dy[1, 3] = INF, float("nan")
    dx, dw = torch.empty_like(x), torch.empty(n, k, device="cuda")
    dgc.linear_backward(dy, x, w, pre, "silu", dx, dw)
    dyd, xd, wd, pred = host(dy, x, w, pre)
    dz = dyd * R.act_pair("silu", pred)[1]
    same_kind("dx", dx, product(dz, wd))
    same_kind("dw", dw, product(dz.t(), xd))
