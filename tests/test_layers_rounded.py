"""The choice of one 16-bit number for dz, as the calls take it, without a GPU."""

import pytest
import torch

from sparsified_gradient_compression_amd import dgc
from test_layers_abi import ECAP, EINVAL, ffn, ffn_backward, linear, linear_backward

ROUNDED = dgc.DGC_DZ_ROUNDED


def test_only_gradients_take_it():
    for act in range(5):
        assert linear(act=act | ROUNDED) == EINVAL and ffn(act=act | ROUNDED) == EINVAL
    for act in (5 | ROUNDED, -1, 2 * ROUNDED, 2 | 2 * ROUNDED):
        assert linear_backward(act=act) == EINVAL and ffn_backward(act=act) == EINVAL


def test_its_workspace_is_its_own():
    """Smaller than the others', and enough for it alone."""
    for fn, call, sizes in ((dgc.dgc_linear_workspace_bytes, linear_backward, (400, 64, 32)),
                            (dgc.dgc_gated_ffn_workspace_bytes, ffn_backward, (400, 32, 64))):
        small, full = fn(*sizes, True, True), fn(*sizes, True)
        assert 0 < small < full and fn(*sizes, False, True) == fn(*sizes, False)
        m, a, b = sizes
        kw = (dict(m=m, n=a, k=b, lddy=a, ldx=b, ldw=b, pre=1 << 20, ldpre=a, lddx=b, lddw=b) if call is linear_backward else
              dict(m=m, d=a, f=b, lddh=b, ldx=a, ldw_gate=a, ldw_up=a, ldgate=b, ldup=b, lddx=a, lddw_gate=a, lddw_up=a))
        assert call(size=full - 1, act=2, **kw) == ECAP and call(size=small - 1, act=2 | ROUNDED, **kw) == ECAP


def test_the_binding_looks_past_it():
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError, match="needs pre"):
        dgc.linear_backward(z(4, 8), z(4, 16), z(8, 16), act="silu", rounded=True)
    with pytest.raises(ValueError, match="on the device of x"):
        dgc.linear_backward(z(4, 8), z(4, 16), z(8, 16), act="none", rounded=True)
