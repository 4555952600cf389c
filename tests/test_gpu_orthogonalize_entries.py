"""orthogonalize entry by entry: remainders of rows and columns, mirrored corners and the last tiles
of each form, which a norm over a whole matrix would let pass."""
import math

import pytest
import torch

import block_ref as R
from test_gpu_orthogonalize import ABC, matrix
from train_ref import half_step

pytestmark = pytest.mark.gpu
L = pytest.importorskip("weight_communication_compression_amd.lowbit")


@pytest.mark.parametrize("steps", [1, 5])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("batch,rows,cols", [
    (1, 2, 3), (1, 65, 63), (2, 128, 512), (1, 100, 5000), (1, 200, 9000), (3, 70, 3000),
    (1, 4100, 64), (2, 640, 640), (1, 1500, 1300), (1, 2100, 2000), (40, 130, 140), (1, 257, 513),
    (2, 777, 1031), (1, 2903, 1031), (1, 129, 127), (1, 1025, 1600)])
def test_every_entry(batch, rows, cols, dtype, steps):
    g = matrix(rows, cols, batch + rows, dtype, batch=(batch,)).cuda()
    out = torch.full(g.shape, math.nan, dtype=torch.bfloat16, device="cuda")
    L.orthogonalize(g, steps=steps, out=out)
    for i in {0, batch // 2, batch - 1}:
        x = g[i].double()
        want = R.newton_schulz(x, steps, ABC, 1e-7, 1.0)
        same = R.newton_schulz(x, steps, ABC, 1e-7, 1.0, R.to_f16)
        # An entry's error is that of many of the operands' roundings to binary16; the largest of all
        # entries with the kernel's roundings is of the size of the largest with the emulated ones.
        # Their 2-norms differ by up to a factor of 2 (binary32 sums turn some roundings the other
        # way), an entry's share of it by as much again.  Then the sums' own 2^-20 and half a
        # step of the result.
        noise = 4 * (same - want).abs().max() + 2 ** -20 * want.abs().max()
        R.close(out[i], want, noise + half_step(torch.bfloat16) * want.abs(), f"{rows} x {cols}, {i}")
        # (and that is well below an entry: what is missing or misplaced shows)
        assert rows * cols < 10 or noise <= 0.2 * want.abs().square().mean().sqrt()
