"""Gradient sets without a single element."""

import pytest
import torch

from sparsified_gradient_compression_amd import dgc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("norm", ("l2", "max"))
@pytest.mark.parametrize("dtypes", ([torch.float32], [torch.bfloat16, torch.float16, torch.float32]))
def test_no_elements(dtypes, norm):
    """Their norm is 0 and their factor `unscale`; there is nothing to write, and a flat gradient of no length."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    grads = [torch.empty(0, 3, dtype=d, device="cuda") for d in dtypes]
    s = dgc.GradSet([g.shape for g in grads], dtypes)
    for call in (lambda: s.pack(grads, torch.empty(0, device="cuda"), 0.5, norm=norm, unscale=0.25),
                 lambda: s.pack(grads, torch.full((4,), 7.0, device="cuda"), 0.5, norm=norm, unscale=0.25),
                 lambda: s.clip(grads, 0.5, norm=norm, unscale=0.25)):
        s.total.fill_(9.0)
        s.scale.fill_(9.0)
        assert float(call()) == 0.0 and float(s.scale) == 0.25
    assert float(s.norm(grads, norm=norm)) == 0.0
