"""Tensors that require a gradient, and what autograd learns of the outputs."""

import pytest
import torch

from sparsified_gradient_compression_amd import dgc

BF16 = torch.bfloat16


def calls(device, grad):
    """Each call with one of its tensors requiring a gradient if `grad`, and what it writes."""
    z = lambda *s, dtype=BF16: torch.zeros(s, dtype=dtype, device=device)  # noqa: E731
    x, w, y, p, q, r = z(4, 16), z(8, 16).requires_grad_(grad), z(4, 8), z(4, 8), z(4, 8), z(4, 8)
    dx, dw, dv, db = z(4, 16), z(8, 16), z(8, 16), z(8)
    return [(lambda: dgc.linear(x, w, out=y, pre=p), [y, p]),
            (lambda: dgc.linear_backward(q, x, w, p, "silu", dx, dw, db), [dx, dw, db]),
            (lambda: dgc.gated_ffn(x, w, w, out=y, gate=p, up=q), [y, p, q]),
            (lambda: dgc.gated_ffn_backward(r, x, w, w, p, q, dx=dx, dw_gate=dw, dw_up=dv), [dx, dw, dv])]


def test_tensors_that_require_a_gradient_are_refused():
    """An output without history would be a gradient of nothing, silently."""
    for i, (call, _) in enumerate(calls("cpu", True)):
        with pytest.raises(ValueError, match="torch.no_grad"):
            call()
            pytest.fail(str(i))
        with torch.no_grad(), pytest.raises(ValueError, match="on the device of x"):  # only the device is wrong
            call()


@pytest.mark.gpu
def test_outputs_know_that_they_were_written():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dgc.lib()
    with torch.no_grad():
        for i, (call, outs) in enumerate(calls("cuda", True)):
            before = [t._version for t in outs]
            call()
            assert all(t._version > b for t, b in zip(outs, before)), i
    g = [torch.ones(5, dtype=BF16, device="cuda"), torch.ones(7, device="cuda")]
    out, flat = [torch.empty_like(t) for t in g], torch.empty(12, device="cuda")
    s = dgc.GradSet([t.shape for t in g], [t.dtype for t in g])
    for call, outs in ((lambda: s.norm(g), [s.total]), (lambda: s.clip(g, 0.5, out=out), out + [s.total, s.scale]),
                       (lambda: s.clip(g, 0.5), g + [s.total, s.scale]), (lambda: s.pack(g, flat, 0.5), [flat, s.total])):
        before = [t._version for t in outs]
        call()
        assert all(t._version > b for t, b in zip(outs, before))
    saved = torch.ones(5, device="cuda", requires_grad=True)
    v = torch.ones(5, device="cuda")
    loss = (saved * v).sum()  # keeps v
    dgc.GradSet([v.shape], [v.dtype]).clip([v], 0.5)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        for call, _ in calls("cuda", False):
            call()
    torch.cuda.synchronize()
