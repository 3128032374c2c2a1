"""Dropout on the GPU: its mask against Philox4x32-10 written out on the host,
its values against the formula, shares that are kept, strides, types, odd
sizes, outputs in the inputs' place, streams, captured calls that draw anew."""

import numpy as np
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


def check_dropout(m, d, dtype, p, residual, pad=0, shift=0, seed=5, offset=0, mk=None):
    mk = mk or Maker(3, pad, shift)
    x = mk.normal(m, d, dtype)
    res = mk.normal(m, d, dtype) if residual else None
    out = mk.empty(m, d, dtype)
    dgc.dropout(x, p, seed, offset, residual=res, out=out)
    torch.cuda.synchronize()
    kept = R.kept(p)
    keep = torch.from_numpy(R.draws(m, d, seed, offset) < kept).cuda()
    y = torch.where(keep, x.double() * (65536 / max(kept, 1)), 0.0)
    e = 2 * R.U * y.abs()  # the factor's rounding and the product's
    if res is not None:
        y = y + res.double()
        e = e + R.U * (y.abs() + res.double().abs())
    R.check("y", out, y, e, dtype)
    dropped = out[~keep]
    assert bool((dropped == (0 if res is None else res[~keep])).all())
    mk.untouched()


SIZES = [(0, 5), (5, 0), (1, 1), (3, 7), (4, 8), (9, 9), (130, 15), (5, 65), (19, 100), (700, 129), (1, 777), (777, 1001),
         (300, 1025), (1, 4096), (65, 4096), (3, 4097), (2, 20001), (5000, 64), (2049, 200), (1, 1000003)]


@pytest.mark.parametrize("m,d", SIZES)
def test_sizes(m, d):
    for dtype, p, residual in ((BF16, 0.1, True), (FP16, 0.5, False), (FP32, 0.9, True), (BF16, 0.0, False)):
        say(f"dropout {m} {d} {dtype} {p} {residual}")
        check_dropout(m, d, dtype, p, residual)


@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (1, 0), (13, 3), (0, 1), (64, 4)])
def test_strides_and_alignment(pad, shift):
    for m, d in ((1, 72), (37, 1001), (130, 264)):
        for dtype in (BF16, FP16, FP32):
            check_dropout(m, d, dtype, 0.3, True, pad, shift)
            check_dropout(m, d, dtype, 0.3, False, pad, shift)


@pytest.mark.parametrize("p", (0.0, 1e-6, 0.25, 0.999, 1 - 2.0 ** -17, 1 - 2.0 ** -18, 1.0))
def test_shares(p):
    check_dropout(33, 500, FP32, p, False)
    check_dropout(33, 500, FP32, p, True)


@pytest.mark.parametrize("seed,offset", [(0, 0), (2 ** 64 - 1, 2 ** 64 - 1), (1 << 32, 1), (7, 1 << 32), (123456789012345678, 98765432109876)])
def test_seeds_and_offsets(seed, offset):
    check_dropout(40, 333, BF16, 0.4, True, seed=seed, offset=offset)


def test_known_words():
    """The published known answers of Philox4x32-10, as the halves they are taken in."""
    for counter, key, want in (((0, 0, 0, 0), (0, 0), "6627e8d5 e169c58d bc57ac4c 9b00dbd8"),
                               ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, "408f276d 41c83b0e a20bc7c6 6d5451fd")):
        got = R.philox([np.array([c], np.uint64) for c in counter], key)
        assert " ".join(f"{int(w[0]):08x}" for w in got) == want


def test_shares_kept_are_as_likely_as_said():
    """The count of kept ones of n draws lies within 6 standard deviations of n K / 65536, in all and by column."""
    m, d, p = 4096, 1024, 0.1
    ones = torch.ones(m, d, dtype=FP32, device="cuda")
    kept = (dgc.dropout(ones, p, 11, 3) > 0).double()
    share = R.kept(p) / 65536
    for total, n in ((kept.sum(), m * d), (kept.sum(0), m), (kept.sum(1), d)):
        assert float((total - n * share).abs().max()) < 6 * (n * share * (1 - share)) ** 0.5
    other = (dgc.dropout(ones, p, 11, 4) > 0).double()
    both = float((kept * other).sum()) - m * d * share * share
    assert abs(both) < 6 * (m * d) ** 0.5 * share


def test_what_is_dropped_counts_as_zero():
    m, d = 30, 200
    keep = torch.from_numpy(R.draws(m, d, 1, 2) < R.kept(0.5)).cuda()
    res = torch.randn(m, d, device="cuda")
    for bad in (float("nan"), float("inf"), -float("inf")):
        x = torch.where(keep, torch.ones_like(res), bad)
        assert bool((dgc.dropout(x, 0.5, 1, 2)[~keep] == 0).all())
        assert torch.equal(dgc.dropout(x, 0.5, 1, 2, residual=res)[~keep], res[~keep])
        x = torch.where(keep, bad, torch.ones_like(res))
        y = dgc.dropout(x, 0.5, 1, 2)
        assert not bool(torch.isfinite(y[keep]).any()) and bool((y[~keep] == 0).all())


def test_gradient():
    """dx = dy * keep / P(keep), also as a difference of sum(dy * y): the map is linear in x, so exact up to roundings."""
    m, d = 50, 333
    x, dy, way = (torch.randn(m, d, device="cuda") for _ in range(3))
    dx = dgc.dropout_backward(dy, 0.3, 9, 1)
    assert torch.equal(dx, dgc.dropout(dy, 0.3, 9, 1))
    f = [float((dy.double() * dgc.dropout(v, 0.3, 9, 1).double()).sum()) for v in (x + way, x)]
    got, size = float((dx.double() * way.double()).sum()), float((dx.abs() * (way.abs() + x.abs())).double().sum())
    assert abs(got - (f[0] - f[1])) < 8 * R.U * size
    inplace = dy.clone()
    assert dgc.dropout_backward(inplace, 0.3, 9, 1, dx=inplace) is inplace and torch.equal(inplace, dx)


def test_outputs_in_the_inputs_place():
    x, res = (torch.randn(77, 301, device="cuda").to(BF16) for _ in range(2))
    want = dgc.dropout(x, 0.2, 4, residual=res)
    for place in (0, 1):
        a = [x.clone(), res.clone()]
        dgc.dropout(a[0], 0.2, 4, residual=a[1], out=a[place])
        assert torch.equal(a[place], want)


def test_streams_and_a_captured_call_that_draws_anew():
    x, res = (torch.randn(77, 1000, device="cuda").to(BF16) for _ in range(2))
    out, step = torch.empty_like(x), torch.zeros(1, dtype=torch.int64, device="cuda")
    s = torch.cuda.Stream()
    want = dgc.dropout(x, 0.2, 4, 1000, residual=res)
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream):
        got = dgc.dropout(x, 0.2, 4, 1000, residual=res, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dgc.dropout(x, 0.2, 4, 990, step=step, residual=res, out=out)
    seen = []
    for i in (0, 10, 3, -1):
        step.fill_(i)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, dgc.dropout(x, 0.2, 4, 990 + i, residual=res)), i
        seen.append(out.clone())
    assert torch.equal(seen[1], want) and not torch.equal(seen[0], seen[1])


def test_rows_far_apart():
    d, ld = 100, (1 << 31) + 8
    buf = torch.empty(2 * ld + d, dtype=BF16, device="cuda")
    x = buf.as_strided((3, d), (ld, 1))
    x.copy_(torch.randn(3, d, device="cuda"))
    want = dgc.dropout(x.contiguous(), 0.5, 3)
    assert torch.equal(dgc.dropout(x, 0.5, 3), want)
    dgc.dropout(x, 0.5, 3, out=x)
    assert torch.equal(x.contiguous(), want)
