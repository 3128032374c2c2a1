"""Where a 16-bit type's precision is lost first: activations far out in their
tails, slopes of the largest values, and the gradients of few rows, whose dz
is kept in two halves."""

import pytest
import torch

import layer_reference as R
from gpu_harness import say
from sparsified_gradient_compression_amd import dgc

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


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


@pytest.mark.parametrize("dtype,low", [(BF16, -12.0), (FP16, -5.0)])
@pytest.mark.parametrize("act", ("silu", "gelu", "gelu_tanh"))
@pytest.mark.parametrize("m", (3, 400))
def test_tails_keep_their_precision(act, dtype, low, m):
    """act(z) and its slope far below 0, relative to themselves: 2^-13 for the
    polynomial of the tail (3e-5) and the rounding of exponents up to 144
    (half a step of binary32 each, five times: 4e-5); a slope's two parts
    cancel to a fifth of either at most in these ranges, and near its zero the
    error is relative to the parts."""
    z = torch.linspace(low, -0.5, m, device="cuda").to(dtype).reshape(m, 1)
    one = torch.ones(1, 1, dtype=dtype, device="cuda")
    y = dgc.linear(z, one, act=act)
    want, slope = R.act_pair(act, z.double())
    if act == "gelu_tanh":  # 1 + tanh cancels in 64 bits too: by the exponential
        q2 = 2 * (2 / torch.pi) ** 0.5 * (z.double() + 0.044715 * z.double() ** 3)
        p = torch.sigmoid(q2)
        want = z.double() * p
        slope = p + want * torch.sigmoid(-q2) * 2 * (2 / torch.pi) ** 0.5 * (1 + 0.134145 * z.double() ** 2)
    R.check("y", y, want, 2.0 ** -13 * want.abs() + 1e-30, dtype)
    dbias = torch.empty(1, dtype=FP32, device="cuda")
    dx = torch.empty_like(z)
    dgc.linear_backward(torch.ones_like(z), z, one, pre=z, act=act, dx=dx, dbias=dbias)
    parts = slope.abs() + 2 * (want / z.double()).abs()  # slope = share + z share'
    e = 2.0 ** -13 * parts + 1e-30
    R.check("dx", dx, slope, e + R.rounding(dtype, slope.abs() + e), dtype)
    R.check("dbias", dbias, slope.sum().reshape(1), e.sum() + R.sum_error(m, slope.abs().sum()), FP32)


@pytest.mark.parametrize("act", ("relu", "silu", "gelu", "gelu_tanh"))
def test_slopes_of_the_largest_values(act):
    big = torch.tensor([1e3, 1e10, 1e20, 1e30, 3e38], device="cuda").to(BF16)
    z = torch.cat([big, -big]).reshape(-1, 1)
    one = torch.ones(1, 1, dtype=BF16, device="cuda")
    dx = torch.empty_like(z)
    dgc.linear_backward(torch.ones_like(z), z, one, pre=z, act=act, dx=dx)
    assert dx.flatten().tolist() == [1.0] * 5 + [0.0] * 5
    y = dgc.linear(z, one, act=act)
    assert torch.equal(y, torch.cat([z[:5], torch.zeros_like(z[5:])]))


def two_halves(dtype, v):
    """How far the sum of two roundings to `dtype` is from v."""
    fi = torch.finfo(dtype)
    return (fi.eps / 2) ** 2 * v.abs() + fi.smallest_normal * fi.eps


# both kernels of every kind: rows on 16 bytes and off them, short and long sums
@pytest.mark.parametrize("m,n,k", [(1, 64, 64), (1, 856, 64), (3, 5, 7), (2, 4096, 200), (17, 520, 1032), (31, 1000, 333),
                                   (32, 8192, 264), (32, 2048, 2056)])
@pytest.mark.parametrize("dtype", (BF16, FP16))
def test_few_rows_keep_dz_in_two_halves(m, n, k, dtype):
    say(f"few rows {m} {n} {k} {dtype}")
    dy, x, pre = normal(1, m, n).to(dtype), normal(2, m, k).to(dtype), normal(3, m, n).to(dtype)
    w = (normal(4, n, k) * k ** -0.5).to(dtype)
    dx, dw = torch.empty_like(x), torch.empty(n, k, device="cuda")
    dgc.linear_backward(dy, x, w, pre, "silu", dx, dw)
    dz, e, _ = R.slope(dy.double(), pre.double(), "silu", dtype)
    e = e + two_halves(dtype, dz.abs() + e)
    R.check("dx", dx, *R.product(dz, w.double(), e, 2 * n), dtype)
    R.check("dw", dw, *R.product(dz.t(), x.double(), e.t(), 2 * m), FP32)
    up, w2 = normal(5, m, n).to(dtype), (normal(6, n, k) * k ** -0.5).to(dtype)
    dg, du = torch.empty(n, k, device="cuda"), torch.empty(n, k, device="cuda")
    dgc.gated_ffn_backward(dy, x, w, w2, pre, up, dx=dx, dw_gate=dg, dw_up=du)
    h, b = dy.double(), up.double()
    value, slope = R.act_pair("silu", pre.double())
    da, db = h * b * slope, h * value
    ea = (h * b).abs() * R.act_error(pre.double(), 0.0) + 2.0 ** -22 * da.abs()
    eb = h.abs() * R.act_error(pre.double(), 0.0) + 2.0 ** -23 * db.abs()
    ea, eb = ea + two_halves(dtype, da.abs() + ea), eb + two_halves(dtype, db.abs() + eb)
    pa, qa = R.product(da, w.double(), ea, 4 * n)
    pb, qb = R.product(db, w2.double(), eb, 4 * n)
    R.check("dx", dx, pa + pb, qa + qb, dtype)
    R.check("dw_gate", dg, *R.product(da.t(), x.double(), ea.t(), 2 * m), FP32)
    R.check("dw_up", du, *R.product(db.t(), x.double(), eb.t(), 2 * m), FP32)


def test_what_overflows_in_the_first_half_has_no_second():
    """dz past fp16's largest value is infinite, as one rounding makes it, and not NaN."""
    dy = torch.full((1, 8), 60000.0, dtype=FP16, device="cuda")
    x, w = torch.ones(1, 8, dtype=FP16, device="cuda"), torch.ones(8, 8, dtype=FP16, device="cuda")
    up, gate = torch.full_like(dy, 4.0), torch.full_like(dy, 20.0)
    dx, dg, du = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    dgc.gated_ffn_backward(dy, x, w, w, gate, up, act="relu", dx=dx, dw_gate=dg, dw_up=du)
    assert bool((dx == float("inf")).all()) and bool((dg == float("inf")).all()) and bool((du == float("inf")).all())
