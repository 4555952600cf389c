"""Host-side checks of what the training-step operators' binding passes on (no GPU
needed)."""
import pytest
import torch

from weight_communication_compression_amd import lowbit as L


def _params(gate, rows_per_gate):
    f = torch.zeros(10, 8)
    return L._join_params(f, f, (("gate", gate),), rows_per_gate, "rms", 1.0, 1e-6, 0.0, 0)


@pytest.mark.parametrize("rows_per_gate", [10, 11, 2 ** 63 - 1, 2 ** 63, 2 ** 64 + 1, 1e30])
def test_the_kernels_take_as_many_rows_a_gate_as_the_check_did(rows_per_gate):
    """One row of the gate for all ten rows: what does not fit 64 bits must not come out as
    fewer rows a gate, whose later rows would be read behind its end."""
    assert _params(torch.ones(1, 8), rows_per_gate).rows_per_gate == 10


def test_a_fraction_counts_as_its_whole_part_in_the_check_too():
    assert _params(torch.ones(5, 8), 2.5).rows_per_gate == 2
    with pytest.raises(L.LowbitError):
        _params(torch.ones(4, 8), 2.5)


@pytest.mark.parametrize("rows_per_gate", [0, -1, 0.5, -2 ** 64 + 3])
def test_gates_of_no_rows_are_refused(rows_per_gate):
    with pytest.raises(L.LowbitError):
        _params(torch.ones(1, 8), rows_per_gate)


def test_inputs_that_require_a_gradient_are_warned_of():
    """The calls stand outside torch's graph of gradients: what is left out of it is said.
    (All of them are refused afterwards, as tensors of the host.)"""
    f, g = torch.zeros(4, 8), torch.zeros(4, 8, requires_grad=True)
    w, t = torch.zeros(5, 8), torch.zeros(4, dtype=torch.int64)
    one = torch.ones(8, requires_grad=True)
    for call in (lambda: L.dropout(g, 0.1, 1),
                 lambda: L.dropout(f, 0.1, 1, residual=g),
                 lambda: L.block_join(g, f), lambda: L.block_join(f, g),
                 lambda: L.block_join(f, f, pre_weight=one),
                 lambda: L.block_join(f, f, gate=one, rows_per_gate=4),
                 lambda: L.linear_xent(g, w, t),
                 lambda: L.linear_xent(f, torch.zeros(5, 8, requires_grad=True), t)):
        with pytest.warns(UserWarning, match="gradient"), pytest.raises(L.LowbitError):
            call()


def test_without_a_graph_of_gradients_nothing_is_warned_of(recwarn):
    f, g = torch.zeros(4, 8), torch.zeros(4, 8, requires_grad=True)
    w, t = torch.zeros(5, 8), torch.zeros(4, dtype=torch.int64)
    with torch.no_grad():
        for call in (lambda: L.dropout(g, 0.1, 1), lambda: L.block_join(g, g, post_weight=g[0]),
                     lambda: L.linear_xent(g, w, t)):
            with pytest.raises(L.LowbitError):
                call()
    for call in (lambda: L.dropout(f, 0.1, 1), lambda: L.block_join(f, f),
                 lambda: L.linear_xent(f, w, t)):
        with pytest.raises(L.LowbitError):
            call()
    assert not recwarn.list
