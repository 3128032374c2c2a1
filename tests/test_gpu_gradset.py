"""Gradient sets on the GPU against 64 bits: norms, clipping in the tensors'
own types, packing into a learner's flat layout."""

import math

import numpy as np
import pytest
import torch

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


def make(seed, sizes, dtypes, shift=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    out = []
    for i, (n, d) in enumerate(zip(sizes, dtypes)):
        at = (shift * (i + 1)) % 9
        buf = torch.full((n + at + 16,), float("nan"), dtype=d, device="cuda")
        buf[at:at + n] = (torch.randn(n, generator=gen, device="cuda") * 10.0 ** (-(i % 4))).to(d)
        out.append(buf[at:at + n])
    return out


def expected(grads, clip, norm, unscale):
    parts = [g.double() for g in grads if g.numel()]
    if norm == "max":
        total = max([float(g.abs().max()) for g in parts], default=0.0)
    else:
        total = math.sqrt(math.fsum(float((g * g).sum()) for g in parts))
    total *= unscale
    return total, unscale * (clip / total if clip > 0 and total > clip else 1.0)


def check_scaled(got, grads, s, dtype):
    """One rounding of the factor, one of the product, one to the type."""
    want = grads.double() * s
    fi = torch.finfo(dtype)
    tol = (2.0 ** -23 + fi.eps / 2) * (1 + 2.0 ** -20) * want.abs() + fi.smallest_normal * fi.eps / 2
    assert got.dtype == dtype
    assert bool(((got.double() - want).abs() <= tol).all())


LAYOUTS = [([1], [BF16]), ([0, 3, 0], [FP32, FP16, BF16]), ([7, 2048, 2049, 1], [FP16, BF16, FP32, FP32]),
           ([100003, 5, 4096 * 9 + 1, 0, 64], [BF16, FP32, FP16, FP16, BF16]),
           ([(i * 37) % 5000 for i in range(1100)], [(BF16, FP16, FP32)[i % 3] for i in range(1100)]),
           ([5_000_001, 3, 2_000_000], [BF16, FP16, FP32])]


@pytest.mark.parametrize("layout", range(len(LAYOUTS)))
@pytest.mark.parametrize("norm", ("l2", "max"))
@pytest.mark.parametrize("shift", (0, 1))
def test_clip_and_pack(layout, norm, shift):
    sizes, dtypes = LAYOUTS[layout]
    grads = make(layout + 10, sizes, dtypes, shift)
    st = dgc.GradSet([(n,) for n in sizes], dtypes)
    for clip, unscale in ((0.5, 1.0), (1e9, 0.125), (0.0, 1.0), (-1.0, 3.0)):
        say(f"layout {layout} {norm} shift {shift} clip {clip} unscale {unscale}")
        total, s = expected(grads, clip, norm, unscale)
        # sums of squares in 64 bits in another order: n * 2^-53 relative, far below this
        tol = 1e-12 * total
        assert abs(float(st.norm(grads, norm=norm, unscale=unscale)) - total) <= tol
        outs = make(99, sizes, dtypes, shift + 2)
        before = [g.clone() for g in grads]
        st.total.fill_(-1)
        assert abs(float(st.clip(grads, clip, out=outs, norm=norm, unscale=unscale)) - total) <= tol
        assert abs(float(st.scale) - s) <= 2.0 ** -24 * s * (1 + 1e-9)
        for g, b, o in zip(grads, before, outs):
            assert torch.equal(g, b)
            check_scaled(o, g, s, g.dtype)
        flat = torch.full((sum(sizes) + 64,), float("nan"), device="cuda")
        st.pack(grads, flat, clip, norm=norm, unscale=unscale)
        assert abs(float(st.total) - total) <= tol
        at = 0
        for g in grads:
            check_scaled(flat[at:at + g.numel()], g, s, FP32)
            at += g.numel()
        assert bool(torch.isnan(flat[at:]).all())
        inplace = [g.clone() for g in grads]
        st.clip(inplace, clip, norm=norm, unscale=unscale)
        assert all(torch.equal(a, b) for a, b in zip(inplace, outs))


def test_nothing_around_the_outputs_is_written():
    sizes, dtypes = [5, 4099, 1], [BF16, FP16, FP32]
    bufs = [torch.full((n + 32,), 7.0, dtype=d, device="cuda") for n, d in zip(sizes, dtypes)]
    outs = [b[9:9 + n] for b, n in zip(bufs, sizes)]
    grads = make(3, sizes, dtypes)
    dgc.GradSet([(n,) for n in sizes], dtypes).clip(grads, 0.1, out=outs)
    for b, n in zip(bufs, sizes):
        assert bool((b[:9] == 7).all()) and bool((b[9 + n:] == 7).all())


def test_large_and_tiny_values_do_not_overflow_the_squares():
    big = [torch.full((1000,), 1e30, device="cuda"), torch.full((10,), 3e38, dtype=BF16, device="cuda")]
    st = dgc.GradSet([g.shape for g in big], [g.dtype for g in big])
    total, s = expected(big, 1.0, "l2", 1.0)
    assert abs(float(st.clip([g.clone() for g in big], 1.0)) - total) <= 1e-12 * total
    tiny = [torch.full((1000,), 1e-30, device="cuda")]
    st = dgc.GradSet([(1000,)], [FP32])
    total, _ = expected(tiny, 1.0, "l2", 1.0)
    assert abs(float(st.norm(tiny)) - total) <= 1e-12 * total


@pytest.mark.parametrize("norm", ("l2", "max"))
def test_zero_infinite_and_nan_gradients(norm):
    g = [torch.zeros(300, device="cuda"), torch.zeros(5000, dtype=BF16, device="cuda")]
    st = dgc.GradSet([t.shape for t in g], [t.dtype for t in g])
    out = [torch.full_like(t, 9.0) for t in g]
    assert float(st.clip(g, 0.5, out=out, norm=norm)) == 0.0 and float(st.scale) == 1.0
    assert all(bool((o == 0).all()) for o in out)
    g[1][4999] = float("inf")
    assert float(st.clip(g, 0.5, out=out, norm=norm)) == math.inf and float(st.scale) == 0.0
    g[0][7] = float("nan")
    g[1][4999] = 2.0
    assert math.isnan(float(st.clip(g, 0.5, out=out, norm=norm))) and float(st.scale) == 1.0


def test_same_results_again_and_on_another_stream():
    sizes, dtypes = LAYOUTS[3]
    grads = make(5, sizes, dtypes)
    st = dgc.GradSet([(n,) for n in sizes], dtypes)
    flat = torch.empty(sum(sizes), device="cuda")
    st.pack(grads, flat, 0.5)
    want, total = flat.clone(), st.total.clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (None, s, s.cuda_stream):
        flat.fill_(float("nan"))
        torch.cuda.synchronize()
        st.pack(grads, flat, 0.5, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(flat, want) and torch.equal(st.total, total)


def test_captured_and_replayed():
    sizes, dtypes = LAYOUTS[4]
    grads = make(6, sizes, dtypes)
    st = dgc.GradSet([(n,) for n in sizes], dtypes)
    flat = torch.empty(sum(sizes), device="cuda")
    st.pack(grads, flat, 0.5)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.pack(grads, flat, 0.5)
    for i in range(4):
        for g, h in zip(grads, make(20 + i, sizes, dtypes)):
            g.copy_(h)
        graph.replay()
        torch.cuda.synchronize()
        got, total = flat.clone(), st.total.clone()
        st.pack(grads, flat, 0.5)
        torch.cuda.synchronize()
        assert torch.equal(got, flat) and torch.equal(total, st.total), i


def test_one_tensor_past_32_bit_offsets():
    n = (1 << 32) + 4099
    g = torch.zeros(n, dtype=BF16, device="cuda")
    g[-1], g[1 << 32], g[0] = 3.0, 4.0, 12.0
    st = dgc.GradSet([(n,)], [BF16])
    flat = torch.empty(n, device="cuda")
    assert float(st.pack([g], flat, 6.5)) == 13.0
    assert [float(flat[i]) for i in (n - 1, 1 << 32, 0, 1)] == [1.5, 2.0, 6.0, 0.0]


def test_packed_gradient_feeds_a_learner():
    """pack and then compress with clip 0 equal one compress of the same
    gradient with its own clip, where both take the same factor."""
    sizes = [4096, 70000, 33]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    grads = [torch.randn(n, generator=gen, device="cuda") for n in sizes]
    k = [max(1, n // 100) for n in sizes]
    flat = torch.empty(sum(sizes), device="cuda")
    dgc.GradSet([(n,) for n in sizes], [FP32] * 3).pack(grads, flat, 0.5)
    a, b = dgc.Learner(sizes, k), dgc.Learner(sizes, k)
    ia, va = a.compress(flat, k, 0.0)
    ib, vb = b.compress(torch.cat(grads), k, 0.5)
    torch.cuda.synchronize()
    assert torch.equal(ia, ib)
    # the two norms' sums differ in order alone: the factor by at most one step
    assert bool(((va - vb).abs() <= 2.0 ** -22 * vb.abs()).all())
    np.testing.assert_allclose(a.v.cpu().numpy(), b.v.cpu().numpy(), rtol=2.0 ** -22)
    a.close()
    b.close()
