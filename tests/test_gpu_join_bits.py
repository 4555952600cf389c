"""GPU checks of the block join: equal calls give equal bits, on any stream, and a row
that its norm cannot take spoils itself alone, in both directions."""
import pytest
import torch

import test_gpu_dropout_join as J
from gpu_util import say
from weight_communication_compression_amd import lowbit as L

pytestmark = pytest.mark.gpu

_device = J._device                      # the module's fixture, for this one too


@pytest.mark.parametrize("rows,cols", [(700, 1032), (900, 40), (33, 4104)])
def test_equal_calls_give_equal_bits_on_any_stream(rows, cols):
    say("equal bits", rows, cols)
    s, how = J.make_join(rows, cols, "bf16", "f32", "f32", "layer", 100, True, 0.1, 1.0, True)
    params = {k: J.gpu(s[k]) for k in J.NAMES}
    f, x, dxo, dz = (J.gpu(s[k]) for k in ("f", "x", "dx_out", "dz"))

    def both():
        out = L.block_join(f, x, **params, **how)
        return (*out, *L.block_join_backward(dxo, dz, f, out.x_out, out.stats, **params, **how))

    ref, again = both(), both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        aside = both()
    torch.cuda.current_stream().wait_stream(side)
    for a, b, c in zip(ref, again, aside):
        assert torch.isfinite(a).all() and torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("cols", [40, 264, 1032, 4104])
def test_a_row_of_zeros_with_eps_0_spoils_itself_alone(cols, norm):
    say("zeros", cols, norm)
    rows, bad = 11, 4
    others = [r for r in range(rows) if r != bad]
    s, how = J.make_join(rows, cols, "bf16", "f32", "f32", norm, 3, True, 0.0, 1.0, True)
    how["eps"] = 0.0
    params = {k: J.gpu(s[k]) for k in J.NAMES}
    f, x, dxo, dz = (J.gpu(s[k]) for k in ("f", "x", "dx_out", "dz"))

    def both():
        out = L.block_join(f, x, **params, **how)
        return out, L.block_join_backward(dxo, dz, f, out.x_out, out.stats, **params, **how)

    clean, clean_back = both()
    f[bad], x[bad] = 0, 0
    out, back = both()
    assert torch.isposinf(out.stats[bad, 1])                  # 1 / sqrt(0)
    for a, b in ((out.x_out, clean.x_out), (out.z, clean.z), (back.df, clean_back.df),
                 (back.dx, clean_back.dx)):
        assert not torch.isfinite(a[bad]).any()               # 0 * infinity
        assert torch.isfinite(a[others]).all() and torch.equal(a[others], b[others])
    # sums over rows: the row's gate group, and every weight that stands with its norms
    assert torch.isfinite(back.dgate[[0, 2, 3]]).all() and torch.isnan(back.dgate[1]).all()
    assert torch.equal(back.dgate[[0, 2, 3]], clean_back.dgate[[0, 2, 3]])
    assert torch.equal(back.dpre_bias, clean_back.dpre_bias)
