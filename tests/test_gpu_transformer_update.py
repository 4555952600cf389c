"""GPU check of the update of examples/train_transformer.py: error feedback through the 4-bit codec
by the oracle, momentum, the orthogonalised update in 64 bits, and the step of every parameter."""
import numpy as np
import pytest
import torch

import block_ref as R
from gpu_util import DEV, say
from test_gpu_transformer_example import example  # noqa: F401  (a fixture)
from train_ref import U, half_step

pytestmark = pytest.mark.gpu


def test_two_updates(example, oracle_mod):  # noqa: F811
    say("transformer update")
    layers, hidden, heads, kv, vocab = 2, 128, 4, 2, 300
    rate, matrix_rate = 0.5, 0.02
    p = example.make_params(layers, hidden, heads, kv, vocab, 5, DEV)
    kinds = ("qkv", "o", "w1", "w2")
    residuals = {n: torch.zeros(v.numel(), device=DEV) for n, v in p.items()}
    momenta = {k: torch.zeros(layers, *p[f"{k}.0"].shape, device=DEV) for k in kinds}
    left = {n: np.zeros(v.numel(), np.float32) for n, v in p.items()}
    moved = {k: torch.zeros(m.shape, dtype=torch.float64) for k, m in momenta.items()}
    half = half_step(torch.bfloat16)
    for turn in range(2):
        g = torch.Generator(device=DEV).manual_seed(turn)
        names = list(p)[::-1]                         # the order of the gradients counts
        grads = {n: torch.randn(p[n].shape, generator=g, device=DEV)
                 .to(torch.float32 if n == "embed" else torch.bfloat16) * 0.1 for n in names}
        before = {n: v.clone() for n, v in p.items()}
        seed = 5000 * turn + 11
        example.apply(p, grads, residuals, momenta, layers, rate, matrix_rate, seed)
        sent = {}
        for i, n in enumerate(names):
            flat = grads[n].float().cpu().numpy().reshape(-1)
            codes, scales, left[n] = oracle_mod.ef_compress(flat, left[n], example.BITS, example.BLOCK,
                                                            True, seed + i, 0)
            back = oracle_mod.unpack_dequant(codes, scales, flat.size, example.BITS, example.BLOCK)
            sent[n] = torch.from_numpy(back).view(p[n].shape)
            assert np.array_equal(residuals[n].cpu().numpy(), left[n]), n
        for n in names:
            kind, _, layer = n.partition(".")
            old, new = before[n].cpu().double(), p[n].cpu().double()
            if kind not in kinds:
                want = old - rate * sent[n].double()
                R.close(new, want, half * want.abs() + 4 * U * (old.abs() + rate * sent[n].abs()), n)
                continue
            at = int(layer)
            moved[kind][at] = 0.9 * moved[kind][at] + sent[n].double()
            m = momenta[kind][at].cpu().double()
            size = moved[kind][at].abs()
            R.close(m, moved[kind][at], 8 * U * (size + 10 * sent[n].abs().max()), f"momentum {n}")
            update = R.newton_schulz(m, 5, (3.4445, -4.7750, 2.0315), 1e-7, 1.0)
            same = R.newton_schulz(m, 5, (3.4445, -4.7750, 2.0315), 1e-7, 1.0, R.to_f16)
            step = matrix_rate * max(1.0, p[n].shape[0] / p[n].shape[1]) ** 0.5
            want = old - step * update
            # the update as test_gpu_orthogonalize_entries.py has it, its step, the parameter's rounding
            off = 4 * (same - update).abs().max() + 2 ** -20 * update.abs().max() + half * update.abs()
            R.close(new, want, step * off + half * (want.abs() + step * off) + 4 * U * old.abs(), n)
            # where the 2-norm of a difference is above that of the bounds, one entry at least is outside
            # its own: no step at all would fail here, and one the other way twice over
            assert (step * update).norm() > 2 * (step * off + half * want.abs()).norm()
