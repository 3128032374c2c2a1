"""Layer norm and its gradients on the GPU against their formulas in 64 bits:
rows of 1 to many thousand columns, no rows, odd sizes, strides and starts,
every type, rows that are constant, far off centre, infinite or NaN, outputs
in the inputs' place, other streams and captured graphs."""

import pytest
import torch

import token_reference as R
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


def wide(t):
    return None if t is None else t.double()


def rows(mk, m, d, dtype, scale=2.0, shift=0.7):
    t = mk.normal(m, d, dtype, scale)
    return t.add_(shift)


def gains(mk, d, kind, dtype):
    """weight and bias: of x's type, in binary32, one of them, none."""
    if kind == "none":
        return None, None
    t = FP32 if kind in ("wide", "weight") else dtype
    w, b = (mk.vector(d, FP32) * 2 + 1).to(t), mk.vector(d, t)
    return (w, None) if kind == "weight" else (None, b) if kind == "bias" else (w, b)


def run_forward(m, d, dtype, kind="own", eps=1e-5, pad=0, shift=0, seed=1, x=None, save=True, **kw):
    mk = Maker(seed, pad, shift)
    x = rows(mk, m, d, dtype) if x is None else x
    w, b = gains(mk, d, kind, dtype)
    out = mk.empty(m, d, dtype)
    mean, rstd = (torch.full((m,), float("nan"), device="cuda") if save else None for _ in range(2))
    dgc.layer_norm(x, w, b, eps=eps, out=out, mean=mean, rstd=rstd, **kw)
    torch.cuda.synchronize()
    if d == 0:  # rows without columns have no mean: nothing is written
        assert not save or bool(torch.isnan(mean).all() and torch.isnan(rstd).all())
        return
    y, ey, mu, emu, r, er = R.layer_norm(x.double(), wide(w), wide(b), eps)
    R.check("y", out, y, ey, dtype)
    if save:
        R.check("mean", mean, mu, emu, FP32)
        R.check("rstd", rstd, r, er, FP32)
    mk.untouched()


def stats(x, eps=1e-5):
    off = x.double() - x.double().mean(1, keepdim=True)
    return x.double().mean(1).float(), ((off * off).mean(1) + eps).rsqrt().float()


def run_backward(m, d, dtype, kind="own", wide_grads=False, residual=True, pad=0, shift=0, seed=2, which="all", **kw):
    mk = Maker(seed, pad, shift)
    x, dy = rows(mk, m, d, dtype), mk.normal(m, d, dtype)
    res = mk.normal(m, d, dtype) if residual else None
    w, _ = gains(mk, d, kind, dtype)
    mean, rstd = stats(x) if m else (torch.empty(0, device="cuda"),) * 2
    g = FP32 if wide_grads else dtype
    dx = mk.empty(m, d, dtype) if which in ("all", "dx") else None
    dw, db = (torch.full((d,), float("nan"), dtype=g, device="cuda") if which in ("all", name) else None
              for name in ("dweight", "dbias"))
    dgc.layer_norm_backward(dy, x, mean, rstd, w, residual=res, dx=dx, dweight=dw, dbias=db, **kw)
    torch.cuda.synchronize()
    if d == 0:
        return
    want = R.layer_norm_backward(dy.double(), x.double(), mean.double(), rstd.double(), wide(w), wide(res))
    for name, got, t in (("dx", dx, dtype), ("dweight", dw, g), ("dbias", db, g)):
        if got is not None:
            R.check(name, got, *want[name], t)
    mk.untouched()


# (m, d): nothing, one element, inside and around the steps of 8, 64, 512, ..., long rows, many rows
SIZES = [(0, 5), (5, 0), (1, 1), (3, 2), (5, 7), (4, 8), (9, 9), (130, 15), (33, 16), (70, 17), (257, 33), (31, 64),
         (5, 65), (19, 100), (64, 127), (700, 129), (3, 255), (9, 257), (2, 511), (33, 512), (7, 513), (1, 777),
         (777, 1000), (2, 1024), (300, 1025), (5, 1152), (1, 2048), (9, 2049), (4, 4095), (1, 4096), (65, 4096),
         (3, 4097), (2, 8191), (17, 8192), (5, 8193), (3, 12288), (2, 16384), (3, 16385), (2, 20001), (1, 65536),
         (3, 70001), (5000, 64), (2049, 200), (1030, 2304), (4100, 1280)]


@pytest.mark.parametrize("m,d", SIZES)
def test_sizes(m, d):
    for dtype, kind in ((BF16, "own"), (FP16, "wide"), (FP32, "own"), (BF16, "none")):
        say(f"layer_norm {m} {d} {dtype} {kind}")
        run_forward(m, d, dtype, kind)
    for dtype, kind, wg, residual in ((BF16, "own", False, True), (FP16, "wide", True, False), (FP32, "own", False, True),
                                      (BF16, "none", True, False)):
        say(f"layer_norm_backward {m} {d} {dtype} {kind} {wg}")
        run_backward(m, d, dtype, kind, wg, residual)


@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (1, 0), (13, 3), (0, 1), (64, 4)])
@pytest.mark.parametrize("m,d", [(1, 72), (37, 1001), (130, 264), (9, 4104), (3, 17000)])
def test_strides_and_alignment(m, d, pad, shift):
    say(f"strides {m} {d} pad {pad} shift {shift}")
    for dtype in (BF16, FP16, FP32):
        run_forward(m, d, dtype, "wide", pad=pad, shift=shift)
        run_backward(m, d, dtype, "wide", True, pad=pad, shift=shift)
    run_forward(m, d, BF16, "weight", pad=pad, shift=shift, save=False)
    run_forward(m, d, FP16, "bias", pad=pad, shift=shift)


@pytest.mark.parametrize("which", ("dx", "dweight", "dbias"))
@pytest.mark.parametrize("m,d", [(40, 1000), (3, 20000), (700, 64)])
def test_one_gradient_alone(m, d, which):
    run_backward(m, d, BF16, "own", which=which)
    run_backward(m, d, FP32, "wide", which=which, residual=False)


@pytest.mark.parametrize("d", (1, 8, 500, 4096, 9000, 20000))
def test_rows_that_are_hard(d):
    """Constant rows, rows far off centre, rows of zeros, tiny and large ones."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(d)
    x = torch.randn(7, d, generator=gen, device="cuda")
    x[0], x[1] = 3.0, 0.0
    x[2] += 1000.0
    x[3] *= 1e-4
    x[4] *= 1e8
    x[5] = x[5] * 30 - 200
    for dtype in (FP32, BF16):
        run_forward(7, d, dtype, "wide", x=x.to(dtype), eps=1e-3)
        run_forward(7, d, dtype, "none", x=x.to(dtype), eps=1e-3)


@pytest.mark.parametrize("d", (5, 1000, 5000, 20000))
def test_infinities_stay_in_their_rows(d):
    x = torch.randn(9, d, device="cuda").to(BF16)
    clean = dgc.layer_norm(x)
    dy = torch.randn(9, d, device="cuda").to(BF16)
    mean, rstd = stats(x)
    dx = torch.empty_like(x)
    dgc.layer_norm_backward(dy, x, mean, rstd, dx=dx)
    bad = x.clone()
    bad[2, d // 2], bad[5, d - 1] = float("inf"), float("nan")
    y = dgc.layer_norm(bad)
    dx2 = torch.empty_like(x)
    dgc.layer_norm_backward(dy, bad, mean, rstd, dx=dx2)
    keep = [0, 1, 3, 4, 6, 7, 8]
    assert torch.equal(y[keep], clean[keep]) and torch.equal(dx2[keep], dx[keep])
    # (n is infinite, and so is the mean of g n: dx is infinite or NaN, by the signs)
    assert bool(torch.isnan(y[[2, 5]]).all()) and not bool(torch.isfinite(dx2[[2, 5]]).any())


@pytest.mark.parametrize("m,d", [(5, 100), (300, 4096), (3, 20000)])
def test_outputs_in_the_inputs_place(m, d):
    mk = Maker(9)
    x, dy, res = rows(mk, m, d, BF16), mk.normal(m, d, BF16), mk.normal(m, d, BF16)
    w, b = gains(mk, d, "own", BF16)
    want = dgc.layer_norm(x, w, b)
    z = x.clone()
    assert dgc.layer_norm(z, w, b, out=z) is z and torch.equal(z, want)
    mean, rstd = stats(x)
    outs = [torch.empty_like(x)] + [torch.empty(d, dtype=BF16, device="cuda") for _ in range(2)]
    dgc.layer_norm_backward(dy, x, mean, rstd, w, res, *outs)
    for place in (0, 1):
        dy2, res2 = dy.clone(), res.clone()
        got = [(dy2, res2)[place]] + [torch.empty(d, dtype=BF16, device="cuda") for _ in range(2)]
        dgc.layer_norm_backward(dy2, x, mean, rstd, w, res2, *got)
        assert all(torch.equal(p, q) for p, q in zip(got, outs)), place


def test_gradients_against_differences():
    """A directional difference of sum(dy * layer_norm(x)) in 64 bits against the gradients, and the same bits each run."""
    m, d = 60, 1000
    mk = Maker(4)
    x, dy = rows(mk, m, d, FP32), mk.normal(m, d, FP32)
    w, b = gains(mk, d, "own", FP32)
    mean, rstd = torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    dgc.layer_norm(x, w, b, mean=mean, rstd=rstd)
    outs = [torch.empty(m, d, device="cuda"), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")]
    dgc.layer_norm_backward(dy, x, mean, rstd, w, None, *outs)
    again = [torch.empty_like(t) for t in outs]
    dgc.layer_norm_backward(dy, x, mean, rstd, w, None, *again)
    assert all(torch.equal(p, q) for p, q in zip(outs, again))
    point = [t.double() for t in (x, w, b)]

    def loss(x, w, b):
        return (dy.double() * R.layer_norm(x, w, b, 1e-5)[0]).sum()

    for i in range(3):
        way = torch.randn(point[i].shape, device="cuda", dtype=torch.float64)
        step = 1e-5
        up, down = list(point), list(point)
        up[i], down[i] = point[i] + step * way, point[i] - step * way
        slope = float((loss(*up) - loss(*down)) / (2 * step))
        got = float((outs[i].double() * way).sum())
        # the difference's own error: step^2 of third derivatives, and 2^-53 * |loss| / step
        scale = float((outs[i].double().abs() * way.abs()).sum())
        assert abs(got - slope) < 1e-4 * scale, (i, got, slope)


def test_streams_and_graphs():
    m, d = 333, 1152
    mk = Maker(8)
    x, dy = rows(mk, m, d, BF16), mk.normal(m, d, BF16)
    w, b = gains(mk, d, "wide", BF16)
    y, mean, rstd = torch.empty_like(x), torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    outs = [torch.empty_like(x), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")]
    space = dgc.layer_norm_workspace(m, d, backward=True)

    def call(stream=None):
        dgc.layer_norm(x, w, b, out=y, mean=mean, rstd=rstd, stream=stream)
        dgc.layer_norm_backward(dy, x, mean, rstd, w, None, *outs, workspace=space, stream=stream)

    def values():
        torch.cuda.synchronize()
        return [t.clone() for t in [y, mean, rstd] + outs]

    call()
    want = values()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        for t in [y, mean, rstd] + outs:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        call(stream)
        assert all(torch.equal(p, q) for p, q in zip(values(), want))
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            call()
    for i in range(4):
        x.add_(0.125 * i)
        graphs[i % 2].replay()
        got = values()
        call()
        assert all(torch.equal(p, q) for p, q in zip(got, values())), i


def test_rows_far_apart():
    """Offsets beyond 2^32 bytes and 2^31 elements."""
    d, ld = 100, (1 << 31) + 8
    buf = torch.empty(2 * ld + d, dtype=BF16, device="cuda")
    x = buf.as_strided((3, d), (ld, 1))
    x.copy_(torch.randn(3, d, device="cuda") + 0.5)
    near = x.contiguous()
    mean, rstd = stats(near)
    dy = torch.randn(3, d, device="cuda").to(BF16)
    want, dwant = dgc.layer_norm(near), torch.empty_like(near)
    dgc.layer_norm_backward(dy, near, mean, rstd, dx=dwant)
    assert torch.equal(dgc.layer_norm(x), want)
    dgc.layer_norm(x, out=x)
    assert torch.equal(x.contiguous(), want)
    x.copy_(near)
    dgc.layer_norm_backward(dy, x, mean, rstd, dx=(dx := torch.empty_like(near)))
    assert torch.equal(dx, dwant)
