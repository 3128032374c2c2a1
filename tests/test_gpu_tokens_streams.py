"""Token operator calls on two streams at once without workspaces of their own,
nothing waited for in between: neither call's memory may be the other's."""

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


def norm_grads(seed):
    m, d = 3000, 1280
    x, dy = normal(seed, m, d), normal(seed + 1, m, d)
    mean, rstd = torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    dgc.layer_norm(x, mean=mean, rstd=rstd)
    w = normal(seed + 2, d)

    def call(stream):
        out = [torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)]
        return dgc.layer_norm_backward(dy, x, mean, rstd, w, None, *out, stream=stream)
    return call


def table_grads(m):
    def of(seed):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        ids = torch.randint(-3, 700, (m,), generator=gen, device="cuda")
        dy = normal(seed, m, 260)

        def call(stream):
            return [dgc.embedding_backward(dy, ids, torch.empty(900, 260, device="cuda"), stream=stream)]
        return call
    return of


def states(ragged):
    def of(seed):
        m, d = 6000, 264
        gate, x, dh = normal(seed, m, d), normal(seed + 1, m, d), normal(seed + 2, m, d)
        rows = {"offsets": torch.tensor([0, 40 + seed, 40 + seed, 5000, m], device="cuda")} if ragged else {"batch": 2}
        n = 4 if ragged else 2
        h = dgc.recurrence(gate, x, **rows)

        def call(stream):
            state, dh0 = torch.empty(n, d, device="cuda"), torch.empty(n, d, device="cuda")
            out = dgc.recurrence(gate, x, out=torch.empty_like(x), state=state, stream=stream, **rows)
            grads = dgc.recurrence_backward(dh, gate, x, h, dgate=torch.empty_like(x), dx=torch.empty_like(x), dh0=dh0,
                                            stream=stream, **rows)
            return [out, state, *grads]
        return call
    return of


@pytest.mark.parametrize("handle", (False, True))
@pytest.mark.parametrize("make", (norm_grads, table_grads(3000), table_grads(30000), states(True), states(False)),
                         ids=("norm", "table", "large table", "ragged", "even"))
def test_calls_without_a_workspace_on_two_streams(make, handle):
    one, two = make(1), make(50)
    want, want2 = one(None), two(None)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(5):
        got = [one(None) for _ in range(3)]
        got2 = two(s.cuda_stream if handle else s)
        got += [one(None)]
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got2, want2)), i
        for g in got:
            assert all(torch.equal(p, q) for p, q in zip(g, want)), i
