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


def test_weights_beyond_32_bits():
    """w and dw of 4.6 GB, a few rows: the far end of both, and dx summed over all of w."""
    n, vocab, hidden, part = 5, 140000, 16384, 10000
    say("xent far weights")
    g = torch.Generator(device=X.DEV)
    g.manual_seed(5)
    x = torch.randn(n, hidden, generator=g, device=X.DEV).bfloat16()
    w = torch.empty(vocab, hidden, dtype=torch.bfloat16, device=X.DEV)
    for a in range(0, vocab, part):
        w[a:a + part] = torch.randn(part, hidden, generator=g, device=X.DEV) * 1.5 / hidden ** 0.5
    t = torch.tensor([0, vocab - 1, 131072, 77, -100], device=X.DEV)
    dloss = torch.full((n,), 0.25, device=X.DEV)
    out = L.linear_xent(x, w, t)
    got = L.linear_xent_backward(x, w, t, out.lse, dloss)
    torch.cuda.synchronize()
    say("  ran")
    x64, counts = x.double(), (t != -100)
    logits = torch.cat([x64 @ w[a:a + part].double().t() for a in range(0, vocab, part)], 1)
    off = (hidden + 1) * X.U * torch.cat([x64.abs() @ w[a:a + part].double().abs().t()
                                          for a in range(0, vocab, part)], 1)
    lse = torch.where(counts, torch.logsumexp(logits, 1), 0.0)
    X.check(out.lse, lse, off.max(1).values + 128 * X.U + 2 * X.U * lse.abs(), "lse")
    d = (logits - out.lse.double()[:, None]).exp() * 0.25
    soft = d.clone()
    rows = torch.arange(4, device=X.DEV)
    d[rows, t[:4]] -= 0.25
    d[4], soft[4] = 0, 0
    half = torch.finfo(torch.bfloat16).eps / 2
    err = soft * (off.exp() - 1 + X.U * (8 + (logits - out.lse.double()[:, None]).abs())) \
        + 4 * X.U * (soft + 0.25 * (d != soft))
    err = err + half * (d.abs() + err)
    for a in (0, 60000, vocab - part):
        want = d[:, a:a + part].t() @ x64
        bound = err[:, a:a + part].t() @ x64.abs() + (n + 4) * X.U * (d[:, a:a + part].t().abs() @ x64.abs())
        X.check(got.dw[a:a + part], want, bound + half * want.abs() + X.TINY * (x64.abs().sum(0) + n + 1),
                "dw")
    want = sum(d[:, a:a + part] @ w[a:a + part].double() for a in range(0, vocab, part))
    bound = sum(err[:, a:a + part] @ w[a:a + part].double().abs()
                + (vocab + 4) * X.U * (d[:, a:a + part].abs() @ w[a:a + part].double().abs())
                for a in range(0, vocab, part))
    X.check(got.dx, want, bound * (1 + 1e-6) + half * want.abs() + X.TINY * vocab, "dx")


def test_tokens_beyond_32_bits():
    """x, its compact copy and dx of 4.8 GB: the far rows equal the same rows alone."""
    n, vocab, hidden = 73000, 300, 32768
    say("xent far tokens")
    g = torch.Generator(device=X.DEV)
    g.manual_seed(6)
    x = torch.empty(n, hidden, dtype=torch.bfloat16, device=X.DEV)
    for a in range(0, n, 1000):
        x[a:a + 1000] = torch.randn(min(1000, n - a), hidden, generator=g, device=X.DEV)
    w = (torch.randn(vocab, hidden, generator=g, device=X.DEV) * 1.5 / hidden ** 0.5).bfloat16()
    t = torch.arange(n, device=X.DEV) % vocab
    t[::3] = -100
    dloss = torch.full((n,), 1e-4, device=X.DEV)
    out = L.linear_xent(x, w, t)
    got = L.linear_xent_backward(x, w, t, out.lse, dloss, need_dw=False)
    torch.cuda.synchronize()
    say("  ran")
    far = slice(n - 500, n)
    X.check_forward(x[far], w, t[far], L.LinearXent(out.loss[far], out.lse[far]))
    X.check_backward(x[far], w, t[far], out.lse[far], dloss[far], None,
                     L.LinearXentGrads(got.dx[far], None))
