"""attention with capped scores where the cap saturates, in both directions, against 64-bit forms."""
import math

import pytest
import torch

import block_ref as R
from test_gpu_attention import BOTH, inputs, offsets, run
from train_ref import U, half_step

pytestmark = pytest.mark.gpu
L = pytest.importorskip("weight_communication_compression_amd.lowbit")


@BOTH
@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("softcap,scale,grow", [(1.0, 20.0, 1.0), (0.5, None, 30.0), (20.0, 150.0, 1.0)])
def test_scores_far_beyond_the_cap(softcap, scale, grow, slopes, dtype):
    """Products of tens to hundreds of times the cap, in whole and in masked tiles."""
    how = dict(dtype=dtype, softcap=softcap, slopes=slopes, scale=scale, grow=grow)
    run([140, 65], heads=4, kv=2, dim=128, **how)
    run([80], [120], causal=False, dim=72, **how)
    run([80, 90], prefix=[30, 90], window=9, **how)
    run([100, 7, 40], [30, 0, 200], heads=4, kv=2, **how)
    run([700, 900], heads=1, **how)                   # keys and queries in parts


@BOTH
@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("softcap", [0.5, 1.0, 4.0])
def test_tanh_over_its_whole_range(softcap, slopes, dtype):
    """Products s, -s and 0 with three keys, s / softcap from 2^-12 to 2^17 in 1024 heads, whose values
    are unit vectors, so that the weights themselves come out."""
    heads = 1024
    x = torch.exp2(torch.linspace(-12, 17, heads)).to(dtype)
    q = torch.zeros(1, heads, 8, dtype=dtype)
    q[0, :, 0] = x
    k, v = torch.zeros(3, 1, 8, dtype=dtype), torch.zeros(3, 1, 8, dtype=dtype)
    for j, s in enumerate((1.0, -1.0, 0.0)):
        k[j, 0, 0], v[j, 0, j] = s, 1.0
    slope = torch.full((heads,), 0.25) if slopes else None
    got = L.attention(q.cuda(), k.cuda(), v.cuda(), scale=softcap, causal=False, softcap=softcap,
                      slopes=None if slope is None else slope.cuda())
    t = torch.tanh(x.double())
    y = softcap * torch.stack([t, -t, torch.zeros_like(t)])
    if slopes:                                        # the query stands at the last key
        y -= 0.25 * torch.tensor([2.0, 1.0, 0.0], dtype=torch.float64)[:, None]
    # The sum and its factor are exact.  A score is off by 8 U softcap and the bias's rounding at
    # most; a weight by twice that, its argument's rounding and a few U of the exp, of
    # the sum and of its reciprocal.
    rel = (16 * softcap + 8 * (softcap + 0.5) + 24) * U
    p = torch.softmax(y, 0)
    weight = 2 * half_step(dtype) if dtype == torch.bfloat16 else half_step(dtype)
    R.close(got.out[0, :, :3].T, p, p * (rel + weight), "weights")
    assert (got.out[0, :, 3:] == 0).all()
    lse = torch.logsumexp(y, 0)
    R.close(got.lse[:, 0], lse, rel + 6 * U * lse.abs() + 6 * U, "lse")


@BOTH
@pytest.mark.parametrize("slopes", [False, True])
def test_unseen_keys_beyond_the_cap(slopes, dtype):
    """Only keys that no query sees saturate, in the same tiles as those that are seen."""
    dim, heads = 64, 2
    q, k, v = inputs([5], [100], heads, 1, dim, dtype, False, 12)
    k[:80] *= 1000
    how = dict(causal=True, window=10, softcap=2.0)
    sl = torch.tensor([0.1, 0.3]) if slopes else None
    call = dict(slopes=None if sl is None else sl.cuda(), **how)
    got = L.attention(q, k, v, **call)
    dout = torch.randn(q.shape, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    grads = L.attention_backward(dout, q, k, v, got.out, got.lse, **call)
    f64 = [t.cpu().double() for t in (q, k, v)]
    at = (offsets([5]), offsets([100]), dim ** -0.5)
    want, err = R.attention(*f64, *at, slopes=sl, dtype=dtype, **how)
    R.close(got.out, want["out"], err["out"], "out")
    R.close(got.lse, want["lse"], err["lse"], "lse")
    want, err = R.attention(*f64, *at, slopes=sl, dtype=dtype, dout=dout.cpu().double(),
                            out=got.out.cpu().double(), lse=got.lse.cpu().double(), **how)
    for n in ("dq", "dk", "dv"):
        R.close(getattr(grads, n), want[n], err[n], n)
    assert (grads.dk[:80] == 0).all() and (grads.dv[:80] == 0).all()


@BOTH
def test_factor_beyond_binary32_of_sums_that_are_not_0(dtype):
    """scale / softcap leaves binary32: every score is +-softcap, here nothing beside 1, and the
    tanh is flat."""
    q, k, v = inputs([70], [70], 2, 1, 64, dtype, False, 13)
    how = dict(causal=False, scale=1.0, softcap=1e-39)
    got = L.attention(q, k, v, **how)
    n = 70
    want = v.double().mean(0).expand(n, 2, 64)
    # weights of 1, exact; a sum of 70 terms, its reciprocal, the result's rounding
    bound = v.double().abs().mean(0) * (n + 4) * U + half_step(dtype) * want.abs()
    R.close(got.out, want, bound.expand(n, 2, 64), "out")
    assert (got.lse.double() - math.log(n)).abs().max() <= 8 * U * math.log(n)
    grads = L.attention_backward(torch.ones_like(q), q, k, v, got.out, got.lse, **how)
    assert (grads.dq == 0).all() and (grads.dk == 0).all()


@BOTH
@pytest.mark.parametrize("softcap", [1e-20, 1e-32, 1e-36])
def test_small_caps_of_small_products(softcap, dtype):
    """Scores that are nothing beside 1, but up to some tens of times their cap: the gradient by q
    knows the difference."""
    run([70, 40], softcap=softcap, scale=1.0, grow=softcap, dtype=dtype)
    run([70, 40], softcap=softcap, scale=0.05, grow=softcap, dtype=dtype, slopes=True)


@BOTH
def test_a_row_beyond_the_cap_changes_no_other(dtype):
    """Waves in which a score comes near the cap take all of theirs another way: to the same bits."""
    q, k, v = inputs([100], [100], 2, 1, 64, dtype, False, 15)
    how = dict(softcap=30.0)
    want = L.attention(q, k, v, **how)
    dout = torch.randn(q.shape, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    grads = L.attention_backward(dout, q, k, v, want.out, want.lse, **how)
    rest = [i for i in range(100) if i != 37]
    q[37] *= 200
    got = L.attention(q, k, v, **how)
    assert torch.equal(got.out[rest], want.out[rest]) and torch.equal(got.lse[:, rest], want.lse[:, rest])
    again = L.attention_backward(dout, q, k, v, got.out, got.lse, **how)
    assert torch.equal(again.dq[rest], grads.dq[rest])
    assert not torch.equal(got.out[37], want.out[37])


@BOTH
def test_nan_stays_nan(dtype):
    q, k, v = inputs([40], [40], 2, 1, 64, dtype, False, 14)
    q[7] = math.nan
    for slopes in (None, torch.full((2,), 0.1, device="cuda")):
        got = L.attention(q, k, v, softcap=1.0, slopes=slopes)
        assert got.out[7].isnan().all() and got.lse[:, 7].isnan().all()
        rest = [i for i in range(40) if i != 7]
        assert not got.out[rest].isnan().any() and not got.lse[:, rest].isnan().any()
