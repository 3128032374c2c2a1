"""Layer and gradient-set calls on two streams at once, nothing waited for in
between: neither call's memory may be the other's."""

import pytest
import torch

from sparsified_gradient_compression_amd import dgc

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dgc.lib()
    return torch


def normal(seed, *shape):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").to(BF16)


@pytest.mark.parametrize("handle", (False, True))
def test_calls_without_a_workspace_on_two_streams(handle):
    m, n, k = 1024, 2048, 1024
    dy, x, pre, w = normal(1, m, n), normal(2, m, k), normal(3, m, n), normal(4, n, k)
    dy2, x2 = normal(5, m, n), normal(6, m, k)

    def grads(dy, x, **kw):
        out = kw.pop("out")
        dgc.linear_backward(dy, x, w, pre, "silu", *out, **kw)

    def new():
        return [torch.empty(s, dtype=BF16, device="cuda") for s in ((m, k), (n, k), (n,))]

    want, want2 = new(), new()
    grads(dy, x, out=want)
    grads(dy2, x2, out=want2)
    y = dgc.linear(x2, w, act="gelu", stream=0)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(5):
        got, got2 = new(), new()
        for _ in range(4):  # its workspace is free again, for this stream, while its kernels run
            grads(dy, x, out=got)
        grads(dy2, x2, out=got2, stream=s.cuda_stream if handle else s)
        y2 = dgc.linear(x2, w, act="gelu", stream=s.cuda_stream if handle else s)
        grads(dy, x, out=got)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got + got2 + [y2], want + want2 + [y])), i


def test_a_set_made_on_one_stream_and_used_on_another():
    sizes = [100003, 5, 70000]
    grads = [normal(i, n) for i, n in enumerate(sizes)]
    flat, flat2 = (torch.empty(sum(sizes), device="cuda") for _ in range(2))
    dgc.GradSet([(n,) for n in sizes], [BF16] * 3).pack(grads, flat, 0.5)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream, 0):
        junk = [torch.full((1 << 20,), 7.0, device="cuda") for _ in range(20)]
        del junk
        st = dgc.GradSet([(n,) for n in sizes], [BF16] * 3, stream=stream)
        st.pack(grads, flat2.fill_(float("nan")), 0.5)
        del st
        torch.cuda.synchronize()
        assert torch.equal(flat, flat2)
