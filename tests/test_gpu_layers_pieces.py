"""The layer gradients to the precision of their own type: behind an activation
dz (da, db) goes to the products as a sum of 16-bit numbers, so that a 16-bit
gradient is off by little more than its one rounding and a binary32 one by
binary32's, at any number of rows; `rounded` asks for one number."""

import pytest
import torch

import layer_reference as R
from gpu_harness import say
from sparsified_gradient_compression_amd import dgc
from test_gpu_layers import Maker

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dgc.lib()
    return torch


def held(dz, e, dtype, pieces, most):
    """The error of dz, e before, as a sum of `pieces` numbers of dtype.  Each but the last leaves at most a step
    (2^-7, 2^-10 of the number), the last at most half a step of what is left: 2^-8 and 2^-16 and 2^-24 (bf16), 2^-11
    and 2^-22 (fp16); the first two of three leave a whole step, 2^-15.  fp16 is scaled: its least number is 2^-24 / 2^14 of the largest |dz|, and two of them may be
    lost (one number: half of one)."""
    bits = {BF16: {1: 8, 2: 16, 3: 24, "2 of 3": 15}, FP16: {1: 11, 2: 22}}[dtype][pieces]
    low = 0.0 if dtype == BF16 else most * (2.0 ** -39 if pieces == 1 else 2.0 ** -37)
    return e + 2.0 ** -bits * (dz.abs() + e) + low


def pieces_of(dtype, wide, rounded, m):
    """(in dx, in dw)"""
    if rounded:
        return (2, 2) if m <= 32 else (1, 1)
    return ("2 of 3", 3) if wide and dtype == BF16 else (2, 2)


def linear(m, n, k, dtype, act, wide, rounded=False, pad=0, shift=0):
    say(f"linear_backward {m} {n} {k} {dtype} {act} wide {wide} rounded {rounded} pad {pad}")
    mk = Maker(2, pad, shift)
    dy, x, w = mk.normal(m, n, dtype), mk.normal(m, k, dtype), mk.normal(n, k, dtype, k ** -0.5)
    pre, g = mk.normal(m, n, dtype), FP32 if wide else dtype
    dx, dw = mk.empty(m, k, dtype), mk.empty(n, k, g)
    ws = dgc.linear_workspace(m, n, k, backward=True, rounded=rounded)
    dgc.linear_backward(dy, x, w, pre=pre, act=act, dx=dx, dw=dw, workspace=ws, rounded=rounded)
    torch.cuda.synchronize()
    dz, e, _ = R.slope(dy.double(), pre.double(), act, dtype)
    most = float(dz.abs().max())
    px, pw = pieces_of(dtype, wide, rounded, m)
    R.check("dx", dx, *R.product(dz, w.double(), held(dz, e, dtype, px, most), 2 * n), dtype)
    R.check("dw", dw, *R.product(dz.t(), x.double(), held(dz, e, dtype, pw, most).t(), pw * m), g)
    mk.untouched()


def gated(m, d, f, dtype, act, wide, rounded=False, pad=0, shift=0):
    say(f"gated_ffn_backward {m} {d} {f} {dtype} {act} wide {wide} rounded {rounded} pad {pad}")
    mk = Maker(4, pad, shift)
    dh, x = mk.normal(m, f, dtype), mk.normal(m, d, dtype)
    wg, wu = mk.normal(f, d, dtype, d ** -0.5), mk.normal(f, d, dtype, d ** -0.5)
    gate, up, g = mk.normal(m, f, dtype), mk.normal(m, f, dtype), FP32 if wide else dtype
    dx, dwg, dwu = mk.empty(m, d, dtype), mk.empty(f, d, g), mk.empty(f, d, g)
    ws = dgc.gated_ffn_workspace(m, d, f, backward=True, rounded=rounded)
    dgc.gated_ffn_backward(dh, x, wg, wu, gate, up, act=act, dx=dx, dw_gate=dwg, dw_up=dwu, workspace=ws,
                           rounded=rounded)
    torch.cuda.synchronize()
    h, a, b = dh.double(), gate.double(), up.double()
    value, slope = R.act_pair(act, a)
    da, db = h * b * slope, h * value
    ea = (h * b).abs() * R.act_error(a, 0.0) + 2.0 ** -22 * da.abs()
    eb = h.abs() * R.act_error(a, 0.0) + 2.0 ** -23 * db.abs()
    most = max(float(da.abs().max()), float(db.abs().max()))
    px, pw = pieces_of(dtype, wide, rounded, m)
    pa, qa = R.product(da, wg.double(), held(da, ea, dtype, px, most), 4 * f)
    pb, qb = R.product(db, wu.double(), held(db, eb, dtype, px, most), 4 * f)
    R.check("dx", dx, pa + pb, qa + qb, dtype)
    R.check("dw_gate", dwg, *R.product(da.t(), x.double(), held(da, ea, dtype, pw, most).t(), pw * m), g)
    R.check("dw_up", dwu, *R.product(db.t(), x.double(), held(db, eb, dtype, pw, most).t(), pw * m), g)
    mk.untouched()


# every kernel: few and many tiles, sums split and not, one step to many, odd numbers of steps, operands off 16 bytes
SIZES = [(1, 64, 72), (7, 35, 70), (32, 72, 264), (33, 72, 264), (64, 200, 72), (70, 72, 8200), (300, 520, 1031), (1000, 264, 520),
         (2000, 2500, 70), (2900, 1352, 3016), (200, 2904, 3016), (1352, 2904, 1528), (515, 1001, 2003)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_linear_backward_is_off_by_its_own_rounding(m, n, k):
    linear(m, n, k, BF16, "gelu_tanh", False)
    linear(m, n, k, FP16, "silu", False)


@pytest.mark.parametrize("m,n,k", SIZES)
def test_gated_ffn_backward_is_off_by_its_own_rounding(m, n, k):
    gated(m, k, n, BF16, "silu", False)
    gated(m, k, n, FP16, "gelu", False)
    gated(m, k, n, BF16, "none", False)


@pytest.mark.parametrize("m,n,k", SIZES)
def test_binary32_weight_gradients_behind_an_activation(m, n, k):
    linear(m, n, k, BF16, "silu", True)
    linear(m, n, k, FP16, "gelu_tanh", True)
    gated(m, k, n, BF16, "gelu", True)
    gated(m, k, n, FP16, "relu", True)


@pytest.mark.parametrize("m,n,k", SIZES)
def test_one_number_where_it_is_asked_for(m, n, k):
    linear(m, n, k, BF16, "silu", True, rounded=True)
    gated(m, k, n, FP16, "silu", False, rounded=True)


@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (13, 3), (64, 4)])
@pytest.mark.parametrize("m,n,k", [(7, 1001, 264), (136, 264, 200), (600, 1032, 328)])
def test_strides_and_alignment(m, n, k, pad, shift):
    linear(m, n, k, BF16, "silu", True, pad=pad, shift=shift)
    gated(m, k, n, BF16, "silu", True, pad=pad, shift=shift)
    gated(m, k, n, FP16, "gelu", False, pad=pad, shift=shift)


def test_relu_keeps_dy_exactly():
    """A slope of 0 or 1 needs no second number: the same as products of dy where pre is above 0."""
    m, n, k = 200, 136, 72
    mk = Maker(6)
    dy, x, w, pre = mk.normal(m, n, BF16), mk.normal(m, k, BF16), mk.normal(n, k, BF16), mk.normal(m, n, BF16)
    a, b = [(torch.empty_like(x), torch.empty(n, k, device="cuda")) for _ in range(2)]
    dgc.linear_backward(dy, x, w, pre, "relu", *a)
    dgc.linear_backward(torch.where(pre > 0, dy, torch.zeros_like(dy)), x, w, None, "none", *b)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_a_workspace_for_rounded_calls_is_refused_elsewhere():
    m, n, k = 200, 136, 72
    mk = Maker(7)
    dy, x, w, pre = mk.normal(m, n, BF16), mk.normal(m, k, BF16), mk.normal(n, k, BF16), mk.normal(m, n, BF16)
    ws = dgc.linear_workspace(m, n, k, backward=True, rounded=True)
    assert ws.numel() < dgc.dgc_linear_workspace_bytes(m, n, k, True)
    with pytest.raises(dgc.DGCError):
        dgc.linear_backward(dy, x, w, pre, "silu", dx=torch.empty_like(x), workspace=ws)
