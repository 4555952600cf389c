"""A call goes to the device that its tensors are on, whatever the current one is (no GPU needed: a
stand-in for the library notes the device that is current when it is called)."""
import contextlib

import pytest
import torch

from weight_communication_compression_amd import lowbit as L

CURRENT, HOST = 3, -1                                 # (host tensors say that they are on device -1)


class Library:
    def __init__(self, real, device):
        self.real, self.device, self.seen, self.status = real, device, [], L.OK

    def __getattr__(self, name):
        if name.endswith("_workspace") or name.startswith("lowbit_num_"):
            return getattr(self.real, name)

        def call(*args):
            assert args[-1] == 100 + HOST            # the handle of the tensors' device's stream
            self.seen.append(self.device[0])
            return self.status
        call.__name__ = name
        return call


@pytest.fixture
def library(monkeypatch):
    device = [CURRENT]
    stand_in = Library(L.lib(), device)

    @contextlib.contextmanager
    def on(d):
        before, device[0] = device[0], d
        try:
            yield
        finally:
            device[0] = before

    monkeypatch.setattr(L, "_lib", stand_in)
    monkeypatch.setattr(L, "_dev", lambda t, what: t.data_ptr())
    monkeypatch.setattr(L, "_gpu", lambda t, what: t.data_ptr())
    monkeypatch.setattr(L, "_raw_stream", lambda d: 100 + d)
    monkeypatch.setattr(L, "_current_device", lambda: device[0])
    monkeypatch.setattr(torch.cuda, "device", on)
    return stand_in


def calls():
    f, x, w = torch.zeros(8, 64), torch.zeros(256), torch.zeros(256, dtype=torch.bfloat16)
    t, one = torch.zeros(8, dtype=torch.int64), torch.zeros(8)
    c = torch.zeros(L.num_words(256, 4), dtype=torch.int32)
    s = torch.zeros(L.num_blocks(256, 64), dtype=torch.float16)
    c32 = torch.zeros(8, dtype=torch.int32)
    q, freqs, lse = torch.zeros(8, 2, 64), torch.zeros(32, dtype=torch.float64), torch.zeros(2, 8)
    return {
        "quantize_pack": lambda: L.quantize_pack(x, 4, 64),
        "unpack_dequant": lambda: L.unpack_dequant(c, s, 256, 4, 64),
        "hadamard_quantize_pack": lambda: L.hadamard_quantize_pack(x, 4, 64),
        "hadamard_unpack_dequant": lambda: L.hadamard_unpack_dequant(c, s, 256, 4, 64),
        "ef_compress": lambda: L.ef_compress(x, x.clone(), 4, 64),
        "ef21_compress": lambda: L.ef21_compress(x, x.clone(), 4, 64),
        "reduce_requant": lambda: L.reduce_requant([c, c], [s, s], 256, 4, 64),
        "reduce_requant_ef": lambda: L.reduce_requant_ef([c, c], [s, s], 256, 4, 64, x.clone()),
        "wdiff_compress": lambda: L.wdiff_compress(w, w, 4, 64),
        "wdiff_apply": lambda: L.wdiff_apply(w, c, s, 4, 64),
        "copy_f32": lambda: L.copy_f32(x, x.clone()),
        "add_inplace_f32": lambda: L.add_inplace_f32(x, x.clone()),
        "fold_f32": lambda: L.fold_f32(x, 4),
        "xor_streams": lambda: L.xor_streams([c32, c32], c32.clone()),
        "dropout": lambda: L.dropout(f, 0.1, 1),
        "dropout_backward": lambda: L.dropout_backward(f, 0.1, 1),
        "block_join": lambda: L.block_join(f, f),
        "block_join_backward": lambda: L.block_join_backward(f, f, f, f, torch.zeros(8, 4)),
        "linear_xent": lambda: L.linear_xent(f, f, t),
        "linear_xent_backward": lambda: L.linear_xent_backward(f, f, t, one, one),
        "rotary": lambda: L.rotary(q, freqs),
        "rotary_backward": lambda: L.rotary_backward(q, freqs),
        "attention": lambda: L.attention(q, q, q),
        "attention_backward": lambda: L.attention_backward(q, q, q, q, q, lse),
        "orthogonalize": lambda: L.orthogonalize(f),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_the_tensors_device_is_the_calls(library, name):
    calls()[name]()
    assert library.seen == [HOST] and library.device == [CURRENT]


@pytest.mark.parametrize("name", ["quantize_pack", "linear_xent", "rotary", "attention"])
def test_a_refused_call_names_itself_and_leaves_the_current_device(library, name):
    library.status = L.EINVAL
    with pytest.raises(L.LowbitError, match=f"lowbit_{name}"):
        calls()[name]()
    assert library.device == [CURRENT]
