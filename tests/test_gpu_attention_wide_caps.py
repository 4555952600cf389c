"""attention with caps far above the scores, whose accuracy must not follow the cap's size, against
64-bit forms."""
import pytest
import torch

import block_ref as R
from test_gpu_attention import BOTH, inputs, offsets
from train_ref import U, half_step

pytestmark = pytest.mark.gpu
L = pytest.importorskip("weight_communication_compression_amd.lowbit")


@BOTH
@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("softcap", [30.0, 512.0, 520.0, 1e4, 1e5, 1e6, 1e9, 1e20, 1e30, 3e38])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** -6])
def test_scores_below_the_cap(scale, softcap, slopes, dtype):
    """Scaled products s, -s and 0 with three keys, s from 2^-6 to 2^5 in 512 heads, whose values are unit
    vectors: weights, lse and gradients as the formula has them."""
    heads = 512
    s = torch.exp2(torch.linspace(-6, 5, heads)).to(dtype)
    q = torch.zeros(1, heads, 8, dtype=dtype)
    q[0, :, 0] = s / scale                             # (exact)
    k, v = torch.zeros(3, heads, 8, dtype=dtype), torch.zeros(3, heads, 8, dtype=dtype)
    for j, sign in enumerate((1.0, -1.0, 0.0)):
        k[j, :, 0], v[j, :, j] = sign, 1.0
    slope = torch.full((heads,), 0.25) if slopes else None
    call = dict(scale=scale, causal=False, softcap=softcap,
                slopes=None if slope is None else slope.cuda())
    cap = float(torch.tensor(softcap))                # as the call passes it on
    t = torch.tanh(s.double() / cap)
    y = cap * torch.stack([t, -t, torch.zeros_like(t)])
    bend = 1 - torch.stack([t, t, torch.zeros_like(t)]) ** 2
    off = 24 * U * y.abs().amax(0)                    # a score is off by 24 U of its own size
    if slopes:                                        # the query stands at the last key
        y = y - 0.25 * torch.tensor([2.0, 1.0, 0.0], dtype=torch.float64)[:, None]
    top = y.abs().amax(0)
    # of a weight: two scores' errors, its argument's and the scores' roundings, a few U of the
    # exp, of the sum and of its reciprocal
    rel = 2 * off + 10 * U * top + 24 * U
    rounded = half_step(dtype) if dtype == torch.bfloat16 else 0.0
    got = L.attention(q.cuda(), k.cuda(), v.cuda(), **call)
    p, lse = torch.softmax(y, 0), torch.logsumexp(y, 0)
    R.close(got.out[0, :, :3].T, p, p * (rel + rounded + half_step(dtype)), "weights")
    R.close(got.lse[:, 0], lse, rel + 6 * U * lse.abs() + 6 * U, "lse")

    dout = torch.randn(1, heads, 8, generator=torch.Generator().manual_seed(1)).to(dtype)
    grads = L.attention_backward(dout.cuda(), q.cuda(), k.cuda(), v.cuda(), got.out, got.lse, **call)
    p = torch.exp(y - got.lse[:, 0].cpu().double())
    d, o = dout[0].double(), got.out[0].cpu().double()
    big = (d * o).abs().sum(1)
    g = p * (d[:, :3].T - (d * o).sum(1)) * bend
    # of g: its weight's error, those of D's sum of eight products and of 1 - tanh^2 (whose tanh is off
    # by 24 U and is below s / softcap)
    goff = g.abs() * rel + p * 12 * U * (d[:, :3].T.abs() + big) + g.abs() * 64 * U
    goff = goff * (1 + rounded) + g.abs() * rounded
    bound = goff[0] + goff[1] + 4 * U * (g[0].abs() + g[1].abs()) \
        + half_step(dtype) * (g[0] - g[1]).abs()
    R.close(grads.dq[0, :, 0], scale * (g[0] - g[1]), scale * bound, "dq")
    for j in range(3):
        want = g[j] * s.double()
        R.close(grads.dk[j, :, 0], want, goff[j] * s.double() + (half_step(dtype) + 4 * U) * want.abs(),
                f"dk of key {j}")
        want = p[j][:, None] * d
        R.close(grads.dv[j], want, want.abs() * (rel + rounded + half_step(dtype) + 4 * U)[:, None],
                f"dv of key {j}")


@BOTH
@pytest.mark.parametrize("slopes", [False, True])
def test_a_cap_that_no_score_comes_near(slopes, dtype):
    """softcap 1e6: the scores are off the uncapped ones by their cube / 3e12 and held to those."""
    for lens, klens, heads, kv, dim, how in (
            ([140, 65], None, 4, 2, 128, dict()),
            ([80], [120], 2, 1, 72, dict(causal=False)),
            ([80, 90], None, 2, 1, 64, dict(prefix=[30, 90], window=9)),
            ([100, 7, 40], [30, 0, 200], 4, 2, 64, dict()),
            ([700, 900], None, 1, 1, 96, dict(window=300)),   # in parts
            ([130], None, 2, 1, 64, dict(scale=-0.3))):
        same, klens = klens is None, klens or lens
        q, k, v = inputs(lens, klens, heads, kv, dim, dtype, same, 21)
        qb, kb = offsets(lens), offsets(klens)
        pre = torch.tensor(how["prefix"], dtype=torch.int32) if "prefix" in how else None
        sl = torch.rand(heads, generator=torch.Generator().manual_seed(7)) * 0.5 if slopes else None
        how = {n: w for n, w in how.items() if n != "prefix"}
        call = dict(q_begin=qb.cuda(), k_begin=None if same else kb.cuda(), softcap=1e6,
                    prefix=None if pre is None else pre.cuda(),
                    slopes=None if sl is None else sl.cuda(), **how)
        how.setdefault("scale", dim ** -0.5)
        f64 = [t.cpu().double() for t in (q, k, v)]
        got = L.attention(q, k, v, **call)
        want, err = R.attention(*f64, qb, kb, prefix=pre, slopes=sl, dtype=dtype, **how)
        R.close(got.out, want["out"], err["out"], f"out {lens}")
        # (the bounds are of products that come with their factor; here a score takes two more
        # roundings and the series' own, of scores of up to 30)
        R.close(got.lse, want["lse"], err["lse"] + 8 * U * 30, f"lse {lens}")
        dout = torch.randn(q.shape, generator=torch.Generator().manual_seed(5)).to(dtype).cuda()
        grads = L.attention_backward(dout, q, k, v, got.out, got.lse, **call)
        want, err = R.attention(*f64, qb, kb, prefix=pre, slopes=sl, dtype=dtype,
                                dout=dout.cpu().double(), out=got.out.cpu().double(),
                                lse=got.lse.cpu().double(), **how)
        for n in ("dq", "dk", "dv"):
            R.close(getattr(grads, n), want[n], err[n], f"{n} {lens}")
