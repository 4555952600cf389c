"""The workspace that a call of the binding allocates lives until the call into the library has
returned, when its kernels have been enqueued (no GPU needed: a stand-in for the library looks)."""
import weakref

import pytest
import torch

from weight_communication_compression_amd import lowbit as L


class Library:
    """Passes on to the library what needs no GPU; of a call with a workspace, notes whether the
    workspace is alive while it runs."""

    def __init__(self, real):
        self.real, self.scratch, self.alive = real, [], []

    def __getattr__(self, name):
        if name.endswith("_workspace"):
            return getattr(self.real, name)

        def call(*args):
            self.alive.append([t() is not None for t in self.scratch])
            return L.OK
        return call


@pytest.fixture
def library(monkeypatch):
    stand_in = Library(L.lib())
    allocate = L._scratch

    def scratch(*args, **named):
        t = allocate(*args, **named)
        stand_in.scratch.append(weakref.ref(t))
        return t

    monkeypatch.setattr(L, "_lib", stand_in)
    monkeypatch.setattr(L, "_scratch", scratch)
    monkeypatch.setattr(L, "_dev", lambda t, what: t.data_ptr())
    monkeypatch.setattr(L, "_gpu", lambda t, what: t.data_ptr())
    monkeypatch.setattr(L, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(L, "_current_device", lambda: -1)       # host tensors'
    return stand_in


def attention(back):
    q, k = torch.zeros(300, 2, 64), torch.zeros(3000, 1, 64)
    if not back:
        return L.attention(q, k, k)
    return L.attention_backward(q, q, k, k, q, torch.zeros(2, 300))


def xent(back):
    x, w, t = torch.zeros(40, 64), torch.zeros(5000, 64), torch.zeros(40, dtype=torch.int64)
    one = torch.zeros(40)
    return L.linear_xent_backward(x, w, t, one, one) if back else L.linear_xent(x, w, t)


def join_backward():
    f = torch.zeros(40, 64)
    return L.block_join_backward(f, f, f, f, torch.zeros(40, 4))


@pytest.mark.parametrize("call", [
    lambda: attention(False), lambda: attention(True), lambda: xent(False), lambda: xent(True),
    join_backward, lambda: L.orthogonalize(torch.zeros(128, 512))],
    ids=["attention", "attention_backward", "linear_xent", "linear_xent_backward",
         "block_join_backward", "orthogonalize"])
def test_the_workspace_outlives_the_call(library, call):
    call()
    assert library.alive == [[True]]


def test_attention_without_parts_takes_none(library):
    q = torch.zeros(3, 2, 64)
    L.attention(q, q, q)
    assert library.alive == [[]]


def test_a_workspace_given_is_used(library):
    q, k = torch.zeros(300, 2, 64), torch.zeros(3000, 1, 64)
    ws = torch.empty(1 << 24, dtype=torch.uint8)
    L.attention(q, k, k, workspace=ws)
    assert library.scratch[0]() is ws
