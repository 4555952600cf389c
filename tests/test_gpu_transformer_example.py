"""GPU checks of examples/train_transformer.py, which runs rotary, attention, block join, linear
xent, the codec and orthogonalize together: its gradients against torch's own differentiation of
the same model in binary32, and that its steps run."""
import importlib.util
import math
import os

import pytest
import torch

import train_ref as R
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LENGTHS = (40, 1, 71, 16)
HEADS, KV = 4, 2


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "train_transformer", os.path.join(ROOT, "examples", "train_transformer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain(p, tokens, targets, layers, drop, seed):
    """The model in binary32, from plain definitions."""
    rows, hidden = tokens.numel(), p["embed"].shape[1]
    dim, factor = hidden // HEADS, R.cut_and_factor(drop)[1]
    at = torch.cat([torch.arange(n) for n in LENGTHS]).to(DEV)
    document = torch.cat([torch.full((n,), i) for i, n in enumerate(LENGTHS)]).to(DEV)
    see = (document[:, None] == document) & (at[:, None] >= at)
    angle = at.double()[:, None] * 10000.0 ** (-2.0 * torch.arange(dim // 2, device=DEV).double() / dim)
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def mask(s, n, cols):
        return torch.from_numpy(R.keep_rows(n, cols, drop, s)).to(DEV) * factor

    def rms(v):
        return v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)

    def turn(t):
        u, v = t.chunk(2, -1)
        return torch.cat([u * c - v * s, u * s + v * c], -1)

    x = z = p["embed"][tokens] * mask(seed, rows, hidden)
    for k in range(layers):
        q, key, val = (z @ p[f"qkv.{k}"].t()).view(rows, -1, dim).split([HEADS, KV, KV], 1)
        q, key = turn(q), turn(key).repeat_interleave(HEADS // KV, 1)
        val = val.repeat_interleave(HEADS // KV, 1)
        scores = (q.transpose(0, 1) @ key.permute(1, 2, 0).contiguous()) / math.sqrt(dim)
        weights = torch.softmax(scores.masked_fill(~see, -math.inf), -1)
        f = (weights @ val.transpose(0, 1).contiguous()).transpose(0, 1).reshape(rows, hidden)
        for block, nth, f in (("a", 0, f @ p[f"o.{k}"].t()), ("f", 1, None)):
            if f is None:
                f = torch.nn.functional.silu(z @ p[f"w1.{k}"].t()) @ p[f"w2.{k}"].t()
            x = x + rms(f) * p[f"post_{block}.{k}"] * mask(seed + 1 + 2 * k + nth, rows, hidden)
            z = rms(x) * p[f"pre_{block}.{k}"]
    return torch.nn.functional.cross_entropy(z @ p["out"].t(), targets, ignore_index=-100)


def test_gradients(example):
    """Against binary32.  A tensor passes about twenty roundings to bfloat16 on its way (each
    step's output, forward and back; two more of the weights of an attention), each off by
    2^-9 in the root mean square: twenty of them by less than 2^-6.8, and the whole
    gradient's relative distance stays within four times 2^-6.8."""
    say("transformer example")
    layers, drop, seed = 2, 0.1, 17
    p = example.make_params(layers, 256, HEADS, KV, 600, 3, DEV)
    rows = sum(LENGTHS)
    tokens = torch.arange(rows, device=DEV) * 5 % 600
    targets = (tokens * 7 + 3) % 600
    targets[::5] = -100
    documents = example.Documents(LENGTHS, 256 // HEADS, DEV)
    loss, grads = example.loss_and_grads(p, tokens, targets, documents, layers, HEADS, KV, drop, seed)
    q = {k: v.float().requires_grad_() for k, v in p.items()}
    want = plain(q, tokens, targets, layers, drop, seed)
    want.backward()
    assert abs(loss.item() - want.item()) <= 2.0 ** -6.8 * abs(want.item())
    for name, v in q.items():
        got = grads[name].float().view(v.shape)
        off = (got - v.grad).norm() / v.grad.norm()
        assert off <= 4 * 2.0 ** -6.8, (name, off.item())


def test_runs(example):
    losses = example.train(steps=3, layers=2, hidden=256, heads=4, kv_heads=2, vocab=512,
                           lengths=(100, 30, 126))
    assert len(losses) == 3 and all(math.isfinite(v) for v in losses)
