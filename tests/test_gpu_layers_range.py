"""Layer gradients in fp16 whose dz (da, db) leaves fp16's range though the
operands and the results do not: products beyond 65504, and below 2^-14, where
fp16 has fewer bits."""

import pytest
import torch

import layer_reference as R
from gpu_harness import say
from sparsified_gradient_compression_amd import dgc

pytestmark = pytest.mark.gpu

FP16, FP32 = torch.float16, torch.float32


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


def held(dz, e, most):
    """dz with its error e, held in fp16 times a power of two that brings the call's largest |dz| to 2^14 at
    least: half a step, or half of fp16's least number, 2^-25 / 2^14 of the largest."""
    return e + 2.0 ** -11 * (dz.abs() + e) + 2.0 ** -39 * most


# (scale of dy, scale of up, scale of w): dz near 2^17 with results below 2^12, near 2^-20 and 2^-24, and near 1
CASES = [(20000.0, 8.0, 2.0 ** -10), (3e-6, 0.25, 1.0), (2.0 ** -12, 2.0 ** -12, 1.0), (1.0, 1.0, 1.0)]


@pytest.mark.parametrize("act", ("silu", "gelu", "relu"))
@pytest.mark.parametrize("m,d,f", [(1, 40, 72), (5, 64, 136), (32, 72, 264), (33, 72, 264), (300, 130, 520), (1030, 264, 35)])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_gated_gradients_out_of_range(m, d, f, act, case):
    sd, su, sw = CASES[case]
    say(f"range {m} {d} {f} {act} case {case}")
    dh, x = (normal(1, m, f) * sd).clamp(-65504, 65504).to(FP16), normal(2, m, d).to(FP16)
    gate, up = normal(3, m, f).to(FP16), (normal(4, m, f) * su).to(FP16)
    wg, wu = ((normal(s, f, d) * f ** -0.5 * sw).to(FP16) for s in (5, 6))
    dx, dg, du = torch.empty_like(x), torch.empty(f, d, device="cuda"), torch.empty(f, d, device="cuda")
    dgc.gated_ffn_backward(dh, x, wg, wu, gate, up, act=act, dx=dx, dw_gate=dg, dw_up=du)
    h, a, b = dh.double(), gate.double(), up.double()
    value, slope = R.act_pair(act, a)
    da, db = h * b * slope, h * value
    most = max(float(da.abs().max()), float(db.abs().max()))
    ea = held(da, (h * b).abs() * R.act_error(a, 0.0) + 2.0 ** -22 * da.abs(), most)
    eb = held(db, h.abs() * R.act_error(a, 0.0) + 2.0 ** -23 * db.abs(), most)
    pa, qa = R.product(da, wg.double(), ea, 4 * f)
    pb, qb = R.product(db, wu.double(), eb, 4 * f)
    R.check("dx", dx, pa + pb, qa + qb, FP16)
    R.check("dw_gate", dg, *R.product(da.t(), x.double(), ea.t(), 2 * m), FP32)
    R.check("dw_up", du, *R.product(db.t(), x.double(), eb.t(), 2 * m), FP32)


@pytest.mark.parametrize("m,n,k", [(1, 64, 64), (4, 35, 70), (32, 264, 72), (40, 264, 72), (700, 136, 264), (70001, 3, 8)])
@pytest.mark.parametrize("scale", (65504.0, 1.0, 1e-6))
def test_linear_gradients_out_of_range(m, n, k, scale):
    """dy up to fp16's largest value under slopes up to 1.13, and next to its least one."""
    say(f"range {m} {n} {k} {scale}")
    dy = (normal(1, m, n) * scale).clamp(-65504, 65504).to(FP16)
    x, pre = normal(2, m, k).to(FP16), normal(3, m, n).to(FP16)
    w = (normal(4, n, k) * 2.0 ** -10).to(FP16)
    dx, dw, db = torch.empty_like(x), torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")
    dgc.linear_backward(dy, x, w, pre, "gelu", dx, dw, db)
    dz, e, _ = R.slope(dy.double(), pre.double(), "gelu", FP16)
    h = held(dz, e, float(dz.abs().max()))
    R.check("dx", dx, *R.product(dz, w.double(), h, 2 * n), FP16)
    R.check("dw", dw, *R.product(dz.t(), x.double(), h.t(), 2 * m), FP32)
    R.check("dbias", db, dz.sum(0), e.sum(0) + R.sum_error(m, dz.abs().sum(0)), FP32)


def test_an_infinite_gradient_does_not_set_the_scale():
    m, n, k = 50, 64, 40
    dy, x, pre, w = (normal(i, *s).to(FP16) for i, s in enumerate(((m, n), (m, k), (m, n), (n, k))))
    dx, dx1 = torch.empty_like(x), torch.empty_like(x)
    dgc.linear_backward(dy, x, w, pre, "silu", dx)
    dy[7, 3], dy[9, 4] = float("inf"), float("nan")
    dgc.linear_backward(dy, x, w, pre, "silu", dx1)
    rows = torch.ones(m, dtype=torch.bool, device="cuda")
    rows[7] = rows[9] = False
    assert torch.equal(dx[rows], dx1[rows]) and bool(torch.isnan(dx1[9]).all()) and not bool(torch.isfinite(dx1[7]).any())


def test_the_scale_is_found_anew_in_every_replay():
    """A captured call on gradients 2^20 times larger and smaller than those it was captured with."""
    m, d, f = 130, 72, 136
    x, dh, gate, up = (normal(i, *s).to(FP16) for i, s in enumerate(((m, d), (m, f), (m, f), (m, f))))
    wg, wu = ((normal(i, f, d) * 2.0 ** -10).to(FP16) for i in (5, 6))
    outs = torch.empty_like(x), torch.empty(f, d, device="cuda"), torch.empty(f, d, device="cuda")
    ws = dgc.gated_ffn_workspace(m, d, f, backward=True)

    def step():
        dgc.gated_ffn_backward(dh, x, wg, wu, gate, up, dx=outs[0], dw_gate=outs[1], dw_up=outs[2], workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i, scale in enumerate((20000.0, 2.0 ** -18, 1.0, 20000.0)):
        dh.copy_((normal(10 + i, m, f) * scale).clamp(-65504, 65504))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) and bool(torch.isfinite(a).all()) for a, b in zip(got, outs)), i


def test_gradients_of_zero_stay_zero():
    m, n, k = 40, 64, 40
    dy, x, pre, w = torch.zeros(m, n, dtype=FP16, device="cuda"), *(normal(i, *s).to(FP16) for i, s in enumerate(((m, k), (m, n), (n, k))))
    dx, dw = torch.full_like(x, 7.0), torch.full_like(w, 7.0)
    dgc.linear_backward(dy, x, w, pre, "silu", dx, dw)
    assert not bool(dx.any()) and not bool(dw.any())
