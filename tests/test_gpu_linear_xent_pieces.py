"""GPU checks of the linear cross entropy and its gradient where rows of w are copied
and the vocabulary is taken in several pieces, in the loss too, against the
64-bit forms and with the bounds of test_gpu_linear_xent (derived there)."""
import pytest
import torch

import test_gpu_linear_xent as X
from gpu_util import DEV, say
from weight_communication_compression_amd import lowbit as L

pytestmark = pytest.mark.gpu

_device = X._device                      # the module's fixture, for this one too

CASES = [  # tokens, vocabulary, hidden, type, pieces
    (20, 70000, 1001, "bf16", 2),
    (20, 40000, 1001, "f32", 2),
    (23, 140000, 1001, "bf16", 3),
    (20, 50257, 1601, "bf16", 2),        # the logits' tiles cut along k
    (512, 50257, 1601, "bf16", 2),
    (130, 65536, 515, "f32", 2),
]


def piece_of(vocab, hidden, dtype):
    """Columns of a piece: copies of up to 128 MiB, equal pieces of whole 256 columns."""
    es = 2 if dtype == "bf16" else 4
    row = -(-hidden * es // 16) * 16
    most = (128 << 20) // row // 256 * 256
    pieces = -(-vocab // most)
    return -(-(-(-vocab // pieces)) // 256) * 256


def scratch(n, vocab, hidden, dtype, back):
    """A workspace in which what is read before it is written shows as NaN."""
    q = L.XentParams(n, vocab, hidden, -100, L.F32 if dtype == "f32" else L.BF16)
    size = L.lib().lowbit_linear_xent_workspace(q, back)
    return torch.full((size,), 255, dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_loss_and_gradient_over_several_pieces(case):
    n, vocab, hidden, dtype, pieces = case
    piece = piece_of(vocab, hidden, dtype)
    assert -(-vocab // piece) == pieces
    say("xent pieces", case, piece)
    x, w, t, dloss, dlse = X.make(n, vocab, hidden, dtype, 0.1)
    edges = [0, vocab - 1, 127, 128, 256]
    for k in range(1, pieces):
        edges += [k * piece + d for d in (-128, -1, 0, 1, 255)]
    edges = [e for e in edges if e < vocab][:n]
    t[:len(edges)] = torch.tensor(edges, device=DEV)
    out = L.linear_xent(x, w, t, workspace=scratch(n, vocab, hidden, dtype, 0))
    torch.cuda.synchronize()
    say("  forward ran")
    X.check_forward(x, w, t, out)
    got = L.linear_xent_backward(x, w, t, out.lse, dloss, dlse=dlse,
                                 workspace=scratch(n, vocab, hidden, dtype, 1))
    torch.cuda.synchronize()
    say("  backward ran")
    X.check_backward(x, w, t, out.lse, dloss, dlse, got)
