"""GPU checks of the block join where rows share a wave, end inside a vector or
take any number of waves, against the 64-bit forms and with the bounds of
test_gpu_dropout_join (derived there)."""
import pytest
import torch

import test_gpu_dropout_join as J
from gpu_util import DEV, say
from weight_communication_compression_amd import lowbit as L

pytestmark = pytest.mark.gpu

_device = J._device                      # the module's fixture, for this one too

CASES = [  # rows, cols, block, stream, params, norm, group (0: no gate), biases, p, a, given
    (70, 5, "bf16", "f32", "f32", "layer", 9, True, 0.3, 1.0, True),     # under one vector
    (1001, 8, "f32", "f32", "f32", "rms", 1, True, 0.1, 1.0, True),
    (1000, 9, "bf16", "bf16", "bf16", "layer", 33, True, 0.2, 0.5, True),  # two vectors, one element
    (1100, 33, "bf16", "bf16", "f32", "rms", 0, True, 0.1, 1.0, True),
    (300, 65, "f32", "f32", "f32", "layer", 300, False, 0.1, 1.0, True),
    (777, 129, "bf16", "f32", "bf16", "rms", 10, True, 0.5, 1.0, True),
    (5000, 255, "f32", "f32", "f32", "layer", 1700, True, 0.0, 0.7, True),
    (513, 500, "bf16", "bf16", "bf16", "rms", 4, False, 0.1, 1.0, True),
    (64, 1027, "bf16", "bf16", "f32", "layer", 5, True, 0.3, 1.0, True),
    (1300, 1540, "bf16", "f32", "f32", "rms", 41, True, 0.1, 1.0, True),
    (37, 3001, "bf16", "bf16", "bf16", "layer", 37, True, 0.2, 1.0, True),
    (1030, 4097, "bf16", "bf16", "bf16", "rms", 3, True, 0.1, 1.0, True),
    (2, 8192, "f32", "f32", "f32", "layer", 1, True, 0.1, 1.0, True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_rows(case):
    J.test_join_and_backward(case)


@pytest.mark.parametrize("cols", [9, 65, 515, 1027, 2051, 4099])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place_where_two_vectors_share_columns(cols, dtype):
    """The last vector of an odd row takes columns of the one before it: outputs that are
    the inputs themselves hold the same bits as outputs of their own."""
    say("in place", cols, dtype)
    s, how = J.make_join(600, cols, dtype, dtype, dtype, "layer", 7, True, 0.2, 0.9, True)
    params = {k: J.gpu(s[k]) for k in J.NAMES}
    f, x, dxo, dz = (J.gpu(s[k]) for k in ("f", "x", "dx_out", "dz"))
    out = L.block_join(f, x, **params, **how)
    ref = L.block_join_backward(dxo, dz, f, out.x_out, out.stats, **params, **how)
    f2, x2 = f.clone(), x.clone()
    L.block_join(f2, x2, x_out=x2, z=f2, **params, **how)
    assert torch.equal(x2, out.x_out) and torch.equal(f2, out.z)
    dxo2, dz2 = dxo.clone(), dz.clone()
    back = L.block_join_backward(dxo2, dz2, f, out.x_out, out.stats, dx=dxo2, df=dz2, **params, **how)
    for a, b in zip(back, ref):
        assert torch.equal(a, b)


@pytest.mark.parametrize("cols", [5, 33, 200, 1029])
def test_nothing_is_written_beside_the_rows(cols):
    """Rows in the middle of a larger buffer: what lies before and behind them stays."""
    rows, guard = 67, 64
    s, how = J.make_join(rows, cols, "bf16", "bf16", "bf16", "rms", 3, False, 0.1, 1.0, True)
    params = {k: J.gpu(s[k]) for k in J.NAMES}
    outs = []
    for _ in range(4):
        whole = torch.full((rows * cols + 2 * guard,), 7.0, dtype=torch.bfloat16, device=DEV)
        outs.append((whole, whole[guard:guard + rows * cols].view(rows, cols)))
    f, x, dxo, dz = (J.gpu(s[k]) for k in ("f", "x", "dx_out", "dz"))
    out = L.block_join(f, x, x_out=outs[0][1], z=outs[1][1], **params, **how)
    L.block_join_backward(dxo, dz, f, out.x_out, out.stats, df=outs[2][1], dx=outs[3][1], **params,
                          **how)
    for whole, inner in outs:
        assert (whole[:guard] == 7).all() and (whole[guard + rows * cols:] == 7).all()
        assert not (inner == 7).all()
