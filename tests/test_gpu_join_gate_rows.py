"""GPU checks of the block join's C entry points where a row of the gate stands for more
rows than there are: the same bits as with exactly as many, into buffers of NaN."""
import ctypes

import pytest
import torch

import test_gpu_dropout_join as J
from gpu_util import DEV, say
from weight_communication_compression_amd import lowbit as L

pytestmark = pytest.mark.gpu

_device = J._device                      # the module's fixture, for this one too


def run(s, rows, cols, rows_per_gate):
    """Forward and backward through the C ABI; all that they write."""
    lib, stream = L.lib(), torch.cuda.current_stream().cuda_stream
    q = L.JoinParams(rows, cols, rows_per_gate, 1, L.BF16, L.F32, L.F32, 1e-5, 0.9, 0.2, 77)
    nan = {k: torch.full(sh, float("nan"), dtype=t, device=DEV) for k, sh, t in
           (("x_out", (rows, cols), torch.float32), ("z", (rows, cols), torch.bfloat16),
            ("stats", (rows, 4), torch.float32), ("df", (rows, cols), torch.bfloat16),
            ("dx", (rows, cols), torch.float32), ("dgate", (1, cols), torch.float32),
            *((k, (cols,), torch.float32) for k in ("dw1", "db1", "dw2", "db2")))}
    p = {k: ctypes.c_void_p(t.data_ptr()) for k, t in {**s, **nan}.items()}
    assert lib.lowbit_block_join(p["f"], p["x"], p["post_weight"], p["post_bias"], p["gate"],
                                 p["pre_weight"], p["pre_bias"], q, p["x_out"], p["z"], p["stats"],
                                 stream) == L.OK
    nbytes = lib.lowbit_block_join_backward_workspace(q)
    ws = torch.full((nbytes,), 255, dtype=torch.uint8, device=DEV)
    assert lib.lowbit_block_join_backward(
        p["dx_out"], p["dz"], p["f"], p["x_out"], p["stats"], p["post_weight"], p["post_bias"],
        p["gate"], p["pre_weight"], q, p["df"], p["dx"], p["dw1"], p["db1"], p["dgate"], p["dw2"],
        p["db2"], ctypes.c_void_p(ws.data_ptr()), nbytes, stream) == L.OK
    torch.cuda.synchronize()
    return nan


@pytest.mark.parametrize("rows,cols", [(1, 40), (2, 520), (3, 64), (9, 1155), (1500, 200)])
def test_one_gate_for_all_rows(rows, cols):
    say("gate rows", rows, cols)
    case = (rows, cols, "bf16", "f32", "f32", "layer", rows, True, 0.2, 0.9, True)
    s = {k: J.gpu(t) for k, t in J.make_join(*case)[0].items()}
    want = run(s, rows, cols, rows)
    for many in (rows + 1, 2 ** 62, 2 ** 63 - rows, 2 ** 63 - 2, 2 ** 63 - 1):
        got = run(s, rows, cols, many)
        for k, t in want.items():
            assert torch.isfinite(t).all() and torch.equal(got[k], t), (k, many)
