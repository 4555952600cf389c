"""GPU checks of the linear cross entropy at sizes where its products' tiles are
whole, cut along k, ragged, or fed from copies of w, against the 64-bit forms and
with the bounds of test_gpu_linear_xent (derived there)."""
import pytest
import torch

import test_gpu_linear_xent as X
from gpu_util import say
from weight_communication_compression_amd import lowbit as L

pytestmark = pytest.mark.gpu

_device = X._device                      # the module's fixture, for this one too

CASES = [
    # tokens, vocabulary, hidden, type, share left out
    (1300, 15000, 2056, "bf16", 0.2),    # 256 x 256 tiles: whole, and cut along k, of logits too
    (1300, 15000, 2056, "bf16", 0.9),    # far fewer rows than the grid is made for
    (2300, 12600, 130, "bf16", 0.1),     # rows of w copied, several rounds of tiles, two steps of k
    (1025, 9001, 1031, "bf16", 0.3),     # odd everything
    (260, 33000, 72, "bf16", 0.0),       # a long sum over the vocabulary for few rows
    (100, 40000, 264, "bf16", 0.1),
    (40, 40000, 520, "bf16", 0.1),
    (1300, 2000, 1040, "f32", 0.2),      # cut along k, of logits too
    (90, 20000, 261, "f32", 0.1),        # rows of w copied
    (19, 2644, 3672, "f32", 0.2),        # the loss cut along k
    (300, 2000, 3001, "bf16", 0.2),      # and with rows of w copied
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_tiles(case):
    n, vocab, hidden, dtype, ignored = case
    say("xent tiles", case)
    x, w, t, dloss, dlse = X.make(n, vocab, hidden, dtype, ignored)
    out = L.linear_xent(x, w, t)
    torch.cuda.synchronize()
    say("  forward ran")
    X.check_forward(x, w, t, out)
    got = L.linear_xent_backward(x, w, t, out.lse, dloss, dlse=dlse)
    torch.cuda.synchronize()
    say("  backward ran")
    X.check_backward(x, w, t, out.lse, dloss, dlse, got)


def test_minus_infinity_beside_a_row_that_ends_inside_a_step():
    """What follows a row of w in memory adds nothing to it, infinite or not."""
    for hidden in (72, 36, 100):
        x, w, t, _, _ = X.make(300, 700, hidden, "bf16", 0.0)
        clean = L.linear_xent(x, w, t)
        w2 = w.clone()
        w2[400, :] = 0
        w2[400, 0] = float("-inf")
        x2 = x.abs()
        one = L.linear_xent(x2, w2, t.clamp(max=399))
        keep = torch.arange(700, device=w.device) != 400
        want = L.linear_xent(x2, w2[keep].contiguous(), t.clamp(max=399))
        assert torch.isfinite(clean.lse).all() and torch.isfinite(one.lse).all(), hidden
        # the same terms, summed in another order: 128 roundings each
        assert ((one.lse - want.lse).abs() <= 2 ** -24 * (256 + 4 * want.lse.abs())).all(), hidden
