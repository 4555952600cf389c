"""What the bindings of rotary, attention and orthogonalize make of numbers that do not fit the C
ABI's fields, and of heads without elements (no GPU needed: a stand-in for the library looks)."""
import pytest
import torch

from weight_communication_compression_amd import lowbit as L


class Library:
    """Passes on to the library what needs no GPU; of the other calls, keeps the parameters."""

    def __init__(self, real):
        self.real, self.params = real, []

    def __getattr__(self, name):
        if name.endswith("_workspace") or name == "lowbit_rotary_frequencies":
            return getattr(self.real, name)

        def call(*args):
            self.params += [a for a in args if isinstance(a, (L.RotaryParams, L.OrthogonalizeParams))]
            return L.OK
        return call


@pytest.fixture
def library(monkeypatch):
    stand_in = Library(L.lib())
    monkeypatch.setattr(L, "_lib", stand_in)
    monkeypatch.setattr(L, "_dev", lambda t, what: t.data_ptr())
    monkeypatch.setattr(L, "_gpu", lambda t, what: t.data_ptr())
    monkeypatch.setattr(L, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(L, "_current_device", lambda: -1)       # host tensors'
    return stand_in


@pytest.mark.parametrize("rows_per_sequence", [10, 11, 2 ** 63, 2 ** 64, 2 ** 64 + 3, 1e30])
def test_as_many_rows_a_sequence_as_there_are(library, rows_per_sequence):
    """Ten rows are one sequence; what does not fit 64 bits must not come out as shorter ones."""
    x, f = torch.zeros(10, 2, 8), torch.zeros(4, dtype=torch.float64)
    L.rotary(x, f, rows_per_sequence=rows_per_sequence)
    L.rotary_backward(x, f, rows_per_sequence=rows_per_sequence)
    assert [p.rows_per_sequence for p in library.params] == [10, 10]


def test_rows_a_sequence_that_fit_are_passed_on(library):
    x, f = torch.zeros(10, 2, 8), torch.zeros(4, dtype=torch.float64)
    L.rotary(x, f, rows_per_sequence=3)
    L.rotary(x, f)
    L.rotary(x[:0], f, rows_per_sequence=3)
    assert [p.rows_per_sequence for p in library.params] == [3, 10, 1]


@pytest.mark.parametrize("rows_per_sequence", [-1, -2 ** 64 + 3])
def test_sequences_of_no_rows_stay_refusable(library, rows_per_sequence):
    L.rotary(torch.zeros(10, 2, 8), torch.zeros(4, dtype=torch.float64),
             rows_per_sequence=rows_per_sequence)
    assert library.params[0].rows_per_sequence < 0


@pytest.mark.parametrize("steps", [65, 2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 64 + 1, -1, -2 ** 32 + 5])
def test_steps_outside_their_range_are_refused(library, steps):
    with pytest.raises(L.LowbitError):
        L.orthogonalize(torch.zeros(4, 4), steps=steps)
    assert not library.params


def test_an_original_length_beyond_64_bits_is_a_long_one():
    far, _ = L.rotary_frequencies(8, scaling="parts", factor=4.0, original_length=2 ** 64 + 5)
    plain, _ = L.rotary_frequencies(8)
    assert torch.equal(far, plain)                    # every pair turns often enough: none is divided
    with pytest.raises(L.LowbitError):
        L.rotary_frequencies(8, scaling="parts", factor=4.0, original_length=-2 ** 64 + 5)


def test_heads_without_elements_are_refused():
    e = torch.zeros(3, 2, 0)
    for call in (lambda: L.attention(e, e, e), lambda: L.attention(e, e, e, scale=1.0),
                 lambda: L.attention_backward(e, e, e, e, e, torch.zeros(2, 3))):
        with pytest.raises(L.LowbitError):
            call()
