"""Embedding and its table's gradient on the GPU against their formulas in 64
bits: no tokens to many, one id for all of them, every id once, padding and
ids out of range, odd widths, strides, types, gradients added to what is there,
the same bits every run, streams and captured graphs."""

import pytest
import torch

import token_reference as R
from gpu_harness import say
from sparsified_gradient_compression_amd import dgc
from test_gpu_layers import Maker

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
I32, I64 = torch.int32, torch.int64


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dgc.lib()
    return torch


def some_ids(m, vocab, kind, dtype, seed=1):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    u = torch.rand(m, generator=gen, device="cuda", dtype=torch.float64)
    if kind == "one":
        ids = torch.full((m,), max(vocab - 1, 0), device="cuda", dtype=I64)
    elif kind == "each":
        ids = torch.randperm(m, generator=gen, device="cuda") % max(vocab, 1)
    elif kind == "zipf":
        ids = (torch.exp(u * torch.log(torch.tensor(vocab + 1.0, dtype=torch.float64, device="cuda"))) - 1).long()
        ids = ids.clamp(0, max(vocab - 1, 0))
    else:  # a third of them padding, far out ones too
        ids = (u * vocab * 1.2).long() - vocab // 6
        ids[: m // 20] = torch.iinfo(dtype).max
        ids[m // 20: m // 10] = torch.iinfo(dtype).min
    return ids.to(dtype)


def known(ids, vocab):
    ids = ids.long()
    return (ids >= 0) & (ids < vocab)


def run_lookup(m, vocab, d, dtype, kind="zipf", itype=I64, scale=1.0, pad=0, shift=0):
    mk = Maker(2, pad, shift)
    table, ids, out = mk.normal(vocab, d, dtype), some_ids(m, vocab, kind, itype), mk.empty(m, d, dtype)
    dgc.embedding(ids, table, scale=scale, out=out)
    torch.cuda.synchronize()
    on = known(ids, vocab)
    want = torch.zeros(m, d, dtype=torch.float64, device="cuda")
    want[on] = table.double()[ids.long()[on]] * scale
    R.check("y", out, want, 2 * R.U * want.abs(), dtype)
    mk.untouched()


def run_backward(m, vocab, d, dtype, kind="zipf", itype=I64, scale=1.0, wide=False, add=False, pad=0, shift=0, **kw):
    mk = Maker(3, pad, shift)
    dy, ids = mk.normal(m, d, dtype), some_ids(m, vocab, kind, itype)
    g = FP32 if wide else dtype
    dtable = mk.empty(vocab, d, g)
    old = None
    if add:
        dtable.copy_(torch.randn(vocab, d, generator=mk.gen, device="cuda"))
        old = dtable.clone()
    dgc.embedding_backward(dy, ids, dtable, scale=scale, accumulate=add, **kw)
    torch.cuda.synchronize()
    on = known(ids, vocab)
    total, size = (torch.zeros(vocab, d, dtype=torch.float64, device="cuda") for _ in range(2))
    total.index_add_(0, ids.long()[on], dy.double()[on])
    size.index_add_(0, ids.long()[on], dy.double().abs()[on])
    # a term goes through at most 32 additions of its unit; units are joined in 64 bits; the scale and its product
    want, e = total * scale, 36 * R.U * size * abs(scale)
    named = torch.zeros(vocab, dtype=torch.bool, device="cuda")
    named[ids.long()[on]] = True
    if add:
        want, e = want + old.double(), e + 2 * R.U * (old.double().abs() + want.abs())
        assert torch.equal(dtable[~named], old[~named])
    else:
        assert bool((dtable[~named] == 0).all())
    R.check("dtable", dtable[named], want[named], e[named], g)
    mk.untouched()


# (m, vocab, d)
SIZES = [(0, 7, 5), (5, 0, 7), (5, 7, 0), (1, 1, 1), (3, 10, 8), (31, 5, 9), (32, 40, 64), (33, 3, 65), (64, 1000, 100),
         (255, 2, 129), (256, 300, 16), (257, 50, 511), (1000, 100, 33), (1023, 2000, 7), (1024, 10, 512),
         (1025, 5000, 40), (2049, 100, 1001), (1531, 10000, 1152), (5000, 33, 72), (32768, 900, 24), (33000, 70000, 12),
         (40000, 3, 8), (2, 8, 20001), (40, 9, 5000), (70000, 200, 2056)]


@pytest.mark.parametrize("m,vocab,d", SIZES)
def test_sizes(m, vocab, d):
    for dtype, kind, itype, scale in ((BF16, "zipf", I64, 1.0), (FP16, "stray", I32, 3.7), (FP32, "each", I64, 0.5),
                                      (BF16, "stray", I64, 8.0)):
        say(f"embedding {m} {vocab} {d} {dtype} {kind} {itype}")
        run_lookup(m, vocab, d, dtype, kind, itype, scale)
    for dtype, kind, itype, scale, wide, add in ((BF16, "zipf", I64, 1.0, True, False), (FP16, "stray", I32, 3.7, False, True),
                                                 (FP32, "one", I64, 0.5, True, False), (BF16, "each", I32, 8.0, False, False),
                                                 (BF16, "one", I64, 1.0, True, True)):
        say(f"embedding_backward {m} {vocab} {d} {dtype} {kind} {itype} {wide} {add}")
        run_backward(m, vocab, d, dtype, kind, itype, scale, wide, add)


@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (1, 0), (13, 3), (0, 1), (64, 4)])
def test_strides_and_alignment(pad, shift):
    for m, vocab, d in ((5, 30, 72), (300, 50, 1001), (130, 1000, 264)):
        for dtype in (BF16, FP16, FP32):
            run_lookup(m, vocab, d, dtype, "stray", I64, 2.0, pad, shift)
            for add in (False, True):
                run_backward(m, vocab, d, dtype, "stray", I32, 2.0, True, add, pad, shift)


@pytest.mark.parametrize("m", (1 << 20, (1 << 20) + 1234))
def test_many_tokens(m):
    """Runs that are merged twice."""
    for kind in ("zipf", "each", "stray"):
        say(f"many tokens {m} {kind}")
        run_backward(m, 300000, 8, BF16, kind, I32, 1.0, True)


def test_large_vocabulary_and_far_offsets():
    """Table rows beyond 2^31 elements and 2^32 bytes."""
    vocab, d = 40_000_000, 64
    table = torch.empty(vocab, d, dtype=BF16, device="cuda")
    ids = torch.tensor([vocab - 1, 0, vocab, vocab - 2, -5, vocab - 1], device="cuda")
    table[ids[[0, 1, 3]]] = torch.randn(3, d, device="cuda").to(BF16)
    y = dgc.embedding(ids, table)
    assert torch.equal(y[[0, 1, 3, 5]], table[ids[[0, 1, 3, 5]]]) and not bool(y[[2, 4]].any())
    dy = torch.randn(6, d, device="cuda").to(BF16)
    dgc.embedding_backward(dy, ids, table)
    assert torch.equal(table[vocab - 1], (dy[0].float() + dy[5].float()).to(BF16))
    assert torch.equal(table[0], dy[1]) and torch.equal(table[vocab - 2], dy[3])
    table[ids[[0, 1, 3]]] = 0
    assert not bool(table.any())


def test_infinities_stay_in_their_rows():
    m, vocab, d = 500, 90, 100
    ids = some_ids(m, vocab, "zipf", I64)
    dy = torch.randn(m, d, device="cuda").to(BF16)
    clean = dgc.embedding_backward(dy, ids, torch.empty(vocab, d, device="cuda"))
    bad = dy.clone()
    bad[77], bad[300] = float("inf"), float("nan")
    got = dgc.embedding_backward(bad, ids, torch.empty(vocab, d, device="cuda"))
    hit = torch.zeros(vocab, dtype=torch.bool, device="cuda")
    hit[ids[[77, 300]]] = True
    assert torch.equal(got[~hit], clean[~hit]) and not bool(torch.isfinite(got[hit]).any())


def test_gradient_against_differences():
    """The look-up is linear in the table: a difference is exact up to the roundings of both."""
    m, vocab, d = 700, 60, 130
    ids = some_ids(m, vocab, "stray", I64)
    table, way = (torch.randn(vocab, d, device="cuda") for _ in range(2))
    dy = torch.randn(m, d, device="cuda")
    f = [float((dy.double() * dgc.embedding(ids, t, scale=3.0).double()).sum()) for t in (table + way, table)]
    dt = dgc.embedding_backward(dy, ids, torch.empty(vocab, d, device="cuda"), scale=3.0)
    size = float((dy.double().abs().sum() * 3 * 6) + 1)
    assert abs(float((dt.double() * way.double()).sum()) - (f[0] - f[1])) < 64 * R.U * size


def test_the_same_bits_every_run_streams_and_graphs():
    m, vocab, d = 5000, 800, 520
    ids = some_ids(m, vocab, "zipf", I32)
    dy = torch.randn(m, d, device="cuda").to(BF16)
    dtable = torch.empty(vocab, d, device="cuda")
    space = dgc.embedding_workspace(m, vocab, d)
    want = dgc.embedding_backward(dy, ids, torch.empty_like(dtable))
    look = dgc.embedding(ids, want.to(BF16), 2.0)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, s, s.cuda_stream):
        got = dgc.embedding_backward(dy, ids, dtable.fill_(float("nan")), stream=stream)
        y = dgc.embedding(ids, want.to(BF16), 2.0) if stream is None else None
        torch.cuda.synchronize()
        assert torch.equal(got, want) and (y is None or torch.equal(y, look))
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            dgc.embedding_backward(dy, ids, dtable, workspace=space)
    for i in range(4):
        ids.copy_(some_ids(m, vocab, ("zipf", "one", "each", "stray")[i], I32, seed=i))
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(dtable, dgc.embedding_backward(dy, ids, torch.empty_like(dtable))), i
