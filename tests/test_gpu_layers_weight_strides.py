"""Gated blocks whose two weights lie in rows of different lengths, one or both
off 16 bytes: the same results as with weights of their own."""

import pytest
import torch

from gpu_harness import say
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


def placed(t, pad, shift):
    """t in rows `pad` elements longer, from element `shift` of a buffer of NaN on."""
    rows, cols = t.shape
    buf = torch.full((rows * (cols + pad) + shift + 8,), float("nan"), dtype=t.dtype, device="cuda")
    out = buf.as_strided((rows, cols), (cols + pad, 1), shift)
    out.copy_(t)
    return out


# few rows (any strides); sizes at which weights are laid out anew; and at which they are read as they are
@pytest.mark.parametrize("m,d,f,as_is", [(5, 1024, 2048, False), (2048, 1024, 4096, False), (70, 136, 200, True)])
@pytest.mark.parametrize("gate,up", [((8, 0), (0, 0)), ((0, 0), (8, 0)), ((8, 0), (16, 0)), ((0, 1), (0, 0)), ((3, 0), (5, 2))])
def test_weights_of_different_strides(m, d, f, as_is, gate, up):
    say(f"weight strides {m} {d} {f} {gate} {up}")
    x, dh, wg, wu = normal(1, m, d), normal(2, m, f), normal(3, f, d) * d ** -0.5, normal(4, f, d) * d ** -0.5

    def run(a, b):
        g, u = torch.empty_like(dh), torch.empty_like(dh)
        h = dgc.gated_ffn(x, a, b, gate=g, up=u)
        dx, dg, du = torch.empty_like(x), torch.empty(f, d, device="cuda"), torch.empty(f, d, device="cuda")
        dgc.gated_ffn_backward(dh, x, a, b, g, u, dx=dx, dw_gate=dg, dw_up=du)
        return h, g, u, dx, dg, du

    # where they are read as they are, by the kernel for rows off 16 bytes
    want = run(placed(wg, 0, 1), placed(wu, 0, 1)) if as_is else run(wg, wu)
    got = run(placed(wg, *gate), placed(wu, *up))
    for name, a, b in zip(("h", "gate", "up", "dx", "dw_gate", "dw_up"), want, got):
        assert torch.equal(a, b), name
