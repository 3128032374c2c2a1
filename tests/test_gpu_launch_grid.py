"""More workgroups than one row of a grid holds: 2^35 gradients, and rows by the
thousand million."""

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
    yield torch
    torch.cuda.empty_cache()


def test_a_set_of_more_than_2_35_gradients():
    n = (1 << 35) + 4099
    say(f"gradient set of {n}")
    g = torch.zeros(n, dtype=BF16, device="cuda")
    at = [0, 1 << 32, 1 << 35, n - 1]
    for i, v in zip(at, (2.0, 4.0, 8.0, 4.0)):
        g[i] = v
    st = dgc.GradSet([(n,)], [BF16])
    assert float(st.clip([g], 5.0)) == 10.0
    assert [float(g[i]) for i in at + [1, 1 << 34]] == [1.0, 2.0, 4.0, 2.0, 0.0, 0.0]


def rows_of(*tensors):
    """The same 2^27 rows of each at a time."""
    return zip(*(t.split(1 << 27) for t in tensors))


def test_rows_by_the_thousand_million():
    """y = x and dx = dy by the identity, dw from the only rows of x that are not 0."""
    m, width = (1 << 30) + 70, 3
    say(f"{m} rows of {width}")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    one = torch.eye(width, dtype=BF16, device="cuda")
    dy = torch.empty(m, width, dtype=BF16, device="cuda")
    for part, in rows_of(dy):
        part.normal_(generator=gen)
    y, dx, dw = torch.empty_like(dy), torch.empty_like(dy), torch.empty(width, width, device="cuda")
    dgc.linear(dy, one, out=y)
    assert all(torch.equal(a, b) for a, b in rows_of(y, dy))
    x = y.zero_()
    rows = [0, (1 << 29) + 3, m - 1]
    for r in rows:
        x[r] = 1.0
    dgc.linear_backward(dy, x, one, dx=dx, dw=dw)
    assert all(torch.equal(a, b) for a, b in rows_of(dx, dy))
    want = dy[rows].float().sum(0)
    assert bool(((dw - want[:, None]).abs() <= 2.0 ** -22 * dy[rows].float().abs().sum(0)[:, None]).all())
    h = dgc.gated_ffn(dx, one, one, act="none", out=y)
    assert all(torch.equal(a, (b.float() * b.float()).to(BF16)) for a, b in rows_of(h, dx))
