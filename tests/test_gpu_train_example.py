"""GPU checks of examples/train_step.py: its gradients against torch's own
differentiation of the same model in binary32, and that a few steps through the
4-bit codec learn."""
import importlib.util
import os

import pytest
import torch

import train_ref as R
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("train_step",
                                                  os.path.join(ROOT, "examples", "train_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain(p, tokens, targets, layers, drop, seed):
    """The model in binary32, its masks from the plain definition."""
    rows, hidden = tokens.numel(), p["embed"].shape[1]
    factor = R.cut_and_factor(drop)[1]

    def mask(s, n, cols):
        return torch.from_numpy(R.keep_rows(n, cols, drop, s)).to(DEV) * factor

    def rms(v):
        return v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)

    x = z = p["embed"][tokens] * mask(seed, rows, hidden)
    for k in range(layers):
        f = torch.nn.functional.silu(z @ p[f"w1.{k}"].t()) @ p[f"w2.{k}"].t()
        x = x + p[f"gate.{k}"] * (rms(f) * p[f"post.{k}"]) * mask(seed + 1 + k, rows, hidden)
        z = rms(x) * p[f"pre.{k}"]
    logits = z @ p["out"].t()
    return torch.nn.functional.cross_entropy(logits, targets, ignore_index=-100)


def test_gradients(example):
    """Against binary32.  A tensor passes about ten roundings to bfloat16 on its way
    (each step's output), each off by at most 2^-8 of a value and by 2^-9 in the root
    mean square: ten of them by less than 2^-7, and the whole gradient's relative
    distance stays within four times that."""
    say("train example")
    layers, drop, seed = 2, 0.1, 17
    p = example.make_params(layers, 256, 600, 3, DEV)
    tokens = torch.arange(96, device=DEV) * 5 % 600
    targets = (tokens * 7 + 3) % 600
    targets[::5] = -100
    loss, grads = example.loss_and_grads(p, tokens, targets, layers, drop, seed)
    q = {k: v.float().requires_grad_() for k, v in p.items()}
    want = plain(q, tokens, targets, layers, drop, seed)
    want.backward()
    assert abs(loss.item() - want.item()) <= 2.0 ** -7 * abs(want.item())
    for name, v in q.items():
        got = grads[name].float().view(v.shape)
        off = (got - v.grad).norm() / v.grad.norm()
        assert off <= 4 * 2.0 ** -7, (name, off.item())


def test_learns(example):
    losses = example.train(steps=12, layers=2, hidden=256, vocab=1024, rows=512)
    assert all(l == l for l in losses)
    assert losses[-1] < 0.9 * losses[0], losses
