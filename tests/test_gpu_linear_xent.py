"""GPU checks of the linear cross entropy and its gradient against plain 64-bit
forms (torch, float64, written out).

Bounds, derived before any run.  A logit is a binary32 sum of `hidden` exact
(bfloat16) or once rounded (binary32) products: off by at most (hidden + 1)
2^-24 sum |x w|.  lse is off by the largest logit error of the row, and its sum of
positive terms by at most 128 roundings of 2^-24 (a lane's terms, the lanes,
the parts).  d = exp(l - lse) (dloss + dlse) - dloss [target] carries the
logit's error, 2^-24 (8 + |l - lse|) and, for bfloat16, half a step of
bfloat16; dx and dw add up d's errors times |w| or |x|, one binary32 rounding of
the running sum for each term, and half a step of their type.  What is below
2^-126 is not held at all."""
import numpy as np
import pytest
import torch

import train_ref as R
from gpu_util import DEV, say
from weight_communication_compression_amd import lowbit as L

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f32": torch.float32}
U = R.U
TINY = 2.0 ** -126                   # smallest normal binary32 and bfloat16


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    L.lib()
    yield
    torch.cuda.synchronize()


def make(n, vocab, hidden, dtype, ignored, seed=0):
    g = np.random.default_rng(n * 1009 + vocab + hidden + seed)
    x = torch.from_numpy(g.standard_normal((n, hidden)).astype(np.float32)).to(T[dtype])
    w = torch.from_numpy((g.standard_normal((vocab, hidden)) * 1.5 / np.sqrt(hidden))
                         .astype(np.float32)).to(T[dtype])
    t = torch.from_numpy(g.integers(0, vocab, n))
    t[torch.from_numpy(g.random(n) < ignored)] = -100
    dloss = torch.from_numpy(g.random(n).astype(np.float32)) / n
    dlse = torch.from_numpy((g.standard_normal(n) / n).astype(np.float32))
    return [v.to(DEV) for v in (x, w, t, dloss, dlse)]


def forward64(x, w, t, ignore=-100):
    """loss, lse, the logits and each row's bound on a logit's error."""
    x, w = x.double(), w.double()
    logits = x @ w.t()
    off = (x.shape[1] + 1) * U * (x.abs() @ w.abs().t())
    top = logits.max(1, keepdim=True).values
    lse = top[:, 0] + (logits - top).exp().sum(1).log()
    rows = torch.arange(len(t), device=DEV)
    hit = logits[rows, t.clamp(0, w.shape[0] - 1)]
    counts = t != ignore
    zero = torch.zeros_like(lse)
    return torch.where(counts, lse - hit, zero), torch.where(counts, lse, zero), logits, off


def check(got, want, bound, what):
    assert got.shape == want.shape, what
    over = ((got.double() - want).abs() / bound.clamp_min(1e-300)).max().item() if got.numel() else 0
    assert over <= 1.0, f"{what}: worst {over:.3g} times the bound"


def check_forward(x, w, t, got):
    loss, lse, logits, off = forward64(x, w, t)
    b = off.max(1).values + 128 * U + 2 * U * lse.abs()
    check(got.lse, lse, b, "lse")
    check(got.loss, loss, 2 * b + 2 * U * loss.abs(), "loss")


def check_backward(x, w, t, lse, dloss, dlse, got):
    dtype = x.dtype
    _, _, logits, off = forward64(x, w, t)
    x64, w64 = x.double(), w.double()
    both = dloss.double() + (0 if dlse is None else dlse.double())
    counts = (t != -100)[:, None]
    gap = logits - lse.double()[:, None]
    soft = torch.where(counts, gap.exp() * both[:, None], 0.0)
    one = torch.zeros_like(soft)
    one[torch.arange(len(t), device=DEV), t.clamp(0)] = dloss.double()
    one = torch.where(counts, one, 0.0)
    d = soft - one
    err = soft.abs() * (off.exp() - 1 + U * (8 + gap.abs())) + 4 * U * (soft.abs() + one.abs())
    if dtype == torch.bfloat16:
        err = err + R.half_step(dtype) * (d.abs() + err)
    n, v = d.shape
    for name, out, a, o in (("dx", got.dx, d, w64), ("dw", got.dw, d.t(), x64)):
        if out is None:
            continue
        e = err if name == "dx" else err.t()
        want = a @ o
        # (d, a product and the result may each be a subnormal and are then lost)
        bound = e @ o.abs() + (a.shape[1] + 4) * U * (a.abs() @ o.abs()) \
            + R.half_step(dtype) * want.abs() + TINY * (o.abs().sum(0) + a.shape[1] + 1)
        check(out, want, bound * (1 + 1e-6), name)


CASES = [(1, 1, 1), (1, 100, 64), (3, 129, 8), (5, 1000, 33), (13, 257, 515), (16, 4099, 128),
         (17, 1000, 64), (40, 700, 200), (130, 300, 72), (129, 1155, 128), (256, 512, 64),
         (255, 1500, 320), (300, 5003, 264), (520, 2049, 96), (700, 1030, 519)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", CASES, ids=lambda c: "x".join(map(str, c)))
def test_forward_and_backward(size, dtype):
    n, vocab, hidden = size
    for ignored, with_lse in ((0.0, False), (0.4, True)):
        say("xent", size, dtype, ignored)
        x, w, t, dloss, dlse = make(n, vocab, hidden, dtype, ignored)
        out = L.linear_xent(x, w, t)
        torch.cuda.synchronize()
        say("  forward ran")
        check_forward(x, w, t, out)
        dlse = dlse if with_lse else None
        got = L.linear_xent_backward(x, w, t, out.lse, dloss, dlse=dlse)
        torch.cuda.synchronize()
        say("  backward ran")
        check_backward(x, w, t, out.lse, dloss, dlse, got)


@pytest.mark.parametrize("dtype,vocab", [("bf16", 4700), ("f32", 2500)])
def test_several_pieces(dtype, vocab):
    """More rows times vocabulary than one piece holds: dx is summed over pieces."""
    x, w, t, dloss, _ = make(60000, vocab, 40, dtype, 0.2)
    say("pieces", dtype)
    out = L.linear_xent(x, w, t)
    got = L.linear_xent_backward(x, w, t, out.lse, dloss)
    for r in range(0, 60000, 20000):
        s = slice(r, r + 20000)
        check_forward(x[s], w, t[s], L.LinearXent(out.loss[s], out.lse[s]))
        check_backward(x[s], w, t[s], out.lse[s], dloss[s], None,
                       L.LinearXentGrads(got.dx[s], None))
    check_backward(x, w, t, out.lse, dloss, None, L.LinearXentGrads(None, got.dw))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nothing_counts_and_no_rows(dtype):
    x, w, t, dloss, _ = make(37, 300, 64, dtype, 0.0)
    t.fill_(-100)
    x[3] = float("nan")                                  # a row that is left out
    out = L.linear_xent(x, w, t)
    assert not out.loss.any() and not out.lse.any()
    got = L.linear_xent_backward(x, w, t, out.lse, dloss)
    assert torch.equal(got.dx, torch.zeros_like(x)) and torch.equal(got.dw, torch.zeros_like(w))
    t[5] = 7
    out = L.linear_xent(x, w, t)
    got = L.linear_xent_backward(x, w, t, out.lse, dloss)
    assert torch.isfinite(got.dw).all() and torch.isfinite(got.dx).all()
    one = L.linear_xent(x[5:6], w, t[5:6])
    assert torch.equal(one.loss, out.loss[5:6])
    empty = L.linear_xent(x[:0], w, t[:0])
    assert empty.loss.shape == (0,)
    got = L.linear_xent_backward(x[:0], w, t[:0], empty.lse, dloss[:0])
    assert got.dx.shape == (0, 64) and torch.equal(got.dw, torch.zeros_like(w))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_infinity_and_bad_targets_stay_in_their_rows(dtype):
    x, w, t, dloss, _ = make(50, 400, 64, dtype, 0.0)
    clean = L.linear_xent(x, w, t)
    bad = x.clone()
    bad[7, 3] = float("nan")
    t2 = t.clone()
    t2[20], t2[21] = 400, -1
    out = L.linear_xent(bad, w, t2)
    for r in range(50):
        if r in (7, 20, 21):
            assert torch.isnan(out.loss[r]) and torch.isnan(out.lse[r])
        else:
            assert torch.equal(out.loss[r], clean.loss[r]) and torch.equal(out.lse[r], clean.lse[r])
    got = L.linear_xent_backward(x, w, t2, clean.lse, dloss)
    assert torch.isnan(got.dx[20]).all() and torch.isnan(got.dx[21]).all()
    assert torch.isfinite(got.dx[:20]).all() and torch.isfinite(got.dx[22:]).all()
    assert torch.isnan(got.dw).all()
    # logits of -infinity count nothing; a row of nothing else has lse -infinity
    x1 = torch.zeros(2, 64, dtype=x.dtype, device=DEV)
    x1[:, 0] = 1
    w1 = torch.zeros(300, 64, dtype=x.dtype, device=DEV)
    w1[:, 0] = float("-inf")
    w1[100:110, 0] = 2.0
    out = L.linear_xent(x1, w1, torch.tensor([100, 105], device=DEV))
    assert torch.allclose(out.lse, torch.full((2,), 2.0 + np.log(10.0), device=DEV), rtol=1e-6)
    w1[100:110, 0] = float("-inf")
    out = L.linear_xent(x1, w1, torch.tensor([100, 105], device=DEV))
    assert torch.equal(out.lse, torch.full((2,), float("-inf"), device=DEV))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_logits_and_uneven_gradients(dtype):
    """Logits of hundreds, d over many orders of magnitude, zero gradients."""
    x, w, t, dloss, _ = make(70, 900, 128, dtype, 0.1)
    x = (x.float() * 60).to(x.dtype)
    dloss = dloss * 10.0 ** -torch.arange(70, device=DEV).float().div(8).floor()
    dloss[11] = 0
    out = L.linear_xent(x, w, t)
    check_forward(x, w, t, out)
    got = L.linear_xent_backward(x, w, t, out.lse, dloss)
    check_backward(x, w, t, out.lse, dloss, None, got)
    zero = L.linear_xent_backward(x, w, t, out.lse, torch.zeros_like(dloss))
    assert not zero.dx.any() and not zero.dw.any()


def test_gradient_against_differences():
    """Of the 64-bit loss, with a weight on lse."""
    x, w, t, dloss, dlse = make(6, 40, 24, "f32", 0.2, seed=3)
    out = L.linear_xent(x, w, t)
    got = L.linear_xent_backward(x, w, t, out.lse, dloss, dlse=dlse)
    v = {"x": x.double(), "w": w.double()}

    def loss():
        a, b, _, _ = forward64(v["x"], v["w"], t)
        return (a * dloss + b * dlse).sum().item()

    for name, grad in (("x", got.dx), ("w", got.dw)):
        flat, g = v[name].view(-1), grad.view(-1)
        for i in range(0, flat.numel(), 17):
            old = flat[i].item()
            flat[i] = old + 1e-5
            a = loss()
            flat[i] = old - 1e-5
            b = loss()
            flat[i] = old
            assert abs((a - b) / 2e-5 - g[i].item()) <= 1e-6, (name, i)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [13, 300])
def test_equal_bits_streams_workspace_and_graph(n, dtype):
    x, w, t, dloss, dlse = make(n, 1100, 136, dtype, 0.3)
    out = L.linear_xent(x, w, t)
    ref = L.linear_xent_backward(x, w, t, out.lse, dloss, dlse=dlse)
    only = L.linear_xent_backward(x, w, t, out.lse, dloss, dlse=dlse, need_dw=False)
    assert only.dw is None and torch.equal(only.dx, ref.dx)
    only = L.linear_xent_backward(x, w, t, out.lse, dloss, dlse=dlse, need_dx=False)
    assert only.dx is None and torch.equal(only.dw, ref.dw)
    q = L.XentParams(n, 1100, 136, -100, L.F32 if dtype == "f32" else L.BF16)
    ws = torch.full((L.lib().lowbit_linear_xent_workspace(q, 1) + 64,), 255, dtype=torch.uint8,
                    device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = L.linear_xent_backward(x, w, t, out.lse, dloss, dlse=dlse, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(again.dx, ref.dx) and torch.equal(again.dw, ref.dw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = L.linear_xent(x, w, t)
        b = L.linear_xent_backward(x, w, t, f.lse, dloss, dlse=dlse)
    for k in range(3):
        for v in (*f, *b):
            v.fill_(float("nan"))
        torch.ones(1000, device=DEV).sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip((*f, *b), (*out, *ref)):
            assert torch.equal(a, c), k
