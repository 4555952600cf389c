"""GPU checks of the linear cross entropy where logits are infinite."""
import pytest
import torch

import test_gpu_linear_xent as X
from weight_communication_compression_amd import lowbit as L

pytestmark = pytest.mark.gpu

_device = X._device                      # the module's fixture, for this one too


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,vocab", [(40, 500), (300, 9000)])
@pytest.mark.parametrize("some", [False, True])
def test_a_logit_of_plus_infinity_spoils_its_row_alone(n, vocab, some, dtype):
    """Every logit of a row, or one among finite ones and logits of -infinity."""
    x, w, t, _, _ = X.make(n, vocab, 64, dtype, 0.0)
    rest = [r for r in range(n) if r != 9]
    x[:, 3] = 0
    w[:, 3] = w[:, 3].abs() + 1
    if some:
        w[:, 3] = -1
        w[77, 3] = 1
    clean = L.linear_xent(x, w, t)
    x[9, 3] = float("inf")
    out = L.linear_xent(x, w, t)
    assert torch.isnan(out.lse[9]) and torch.isnan(out.loss[9])
    assert torch.isfinite(clean.lse).all()
    assert torch.equal(out.lse[rest], clean.lse[rest])
    assert torch.equal(out.loss[rest], clean.loss[rest])
