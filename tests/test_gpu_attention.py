"""attention and its gradient against 64-bit forms."""
import math

import pytest
import torch

import block_ref as R

pytestmark = pytest.mark.gpu
L = pytest.importorskip("weight_communication_compression_amd.lowbit")


def offsets(lens, first=0):
    b = [first]
    for n in lens:
        b.append(b[-1] + n)
    return torch.tensor(b, dtype=torch.int32)


def inputs(lens, klens, heads, kv, dim, dtype, packed, seed, first=0, behind=0):
    g = torch.Generator().manual_seed(seed)
    tq, tk = first + sum(lens) + behind, first + sum(klens) + behind
    if packed:
        qkv = torch.randn(tq, heads + 2 * kv, dim, generator=g).to(dtype).cuda()
        return qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    return tuple(torch.randn(t, n, dim, generator=g).to(dtype).cuda()
                 for t, n in ((tq, heads), (tk, kv), (tk, kv)))


def run(lens, klens=None, heads=2, kv=1, dim=64, dtype=torch.bfloat16, causal=True, window=0,
        prefix=None, softcap=0.0, slopes=False, packed=None, seed=0, scale=None, grow=1.0):
    """Both directions against the 64-bit forms; the outputs."""
    same = klens is None
    klens = lens if same else klens
    q, k, v = inputs(lens, klens, heads, kv, dim, dtype, same if packed is None else packed, seed)
    q = q * grow if grow != 1.0 else q
    qb, kb = offsets(lens), offsets(klens)
    pre = None if prefix is None else torch.tensor(prefix, dtype=torch.int32)
    sl = torch.rand(heads, generator=torch.Generator().manual_seed(7)) * 0.5 if slopes else None
    how = dict(scale=scale, causal=causal, window=window, softcap=softcap)
    call = dict(q_begin=qb.cuda(), k_begin=None if same else kb.cuda(),
                prefix=None if pre is None else pre.cuda(), slopes=None if sl is None else sl.cuda(),
                **how)
    how["scale"] = dim ** -0.5 if scale is None else scale
    what = f"{lens} {klens} {heads}/{kv} {dim} {dtype} {how} {prefix}"
    got = L.attention(q, k, v, **call)
    f64 = [t.cpu().double() for t in (q, k, v)]
    want, err = R.attention(*f64, qb, kb, prefix=pre, slopes=sl, dtype=dtype, **how)
    R.close(got.out, want["out"], err["out"], "out " + what)
    R.close(got.lse, want["lse"], err["lse"], "lse " + what)
    dout = torch.randn(q.shape, generator=torch.Generator().manual_seed(seed + 1)).to(dtype).cuda()
    grads = L.attention_backward(dout, q, k, v, got.out, got.lse, **call)
    want, err = R.attention(*f64, qb, kb, prefix=pre, slopes=sl, dtype=dtype, dout=dout.cpu().double(),
                            out=got.out.cpu().double(), lse=got.lse.cpu().double(), **how)
    for n in ("dq", "dk", "dv"):
        R.close(getattr(grads, n), want[n], err[n], f"{n} {what}")
    return got, grads


BOTH = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])


@BOTH
@pytest.mark.parametrize("n", [1, 2, 31, 33, 63, 64, 65, 127, 128, 129, 200, 257])
def test_lengths(n, dtype):
    run([n], dtype=dtype, dim=64, causal=True)
    run([n], dtype=dtype, dim=128, causal=False, heads=1)


@BOTH
@pytest.mark.parametrize("dim", [8, 16, 24, 40, 72, 80, 96, 104, 120, 128])
def test_head_dims(dim, dtype):
    run([70, 40], dim=dim, dtype=dtype, heads=3, kv=3)


@BOTH
@pytest.mark.parametrize("heads,kv", [(1, 1), (4, 1), (6, 2), (8, 8), (5, 5), (16, 8), (24, 12)])
def test_shared_heads(heads, kv, dtype):
    run([90, 1, 0, 37], heads=heads, kv=kv, dtype=dtype, dim=64)


@BOTH
def test_documents(dtype):
    run([0, 5, 130, 0, 0, 1, 64, 1, 1, 129, 0], dtype=dtype)
    run([3] * 70, dtype=dtype, heads=1)               # more than 64 sequences
    run([1] * 200 + [0] * 10 + [40], dtype=dtype, heads=1, causal=False)


@BOTH
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [1, 2, 17, 64, 100, 1000])
def test_windows(window, causal, dtype):
    run([150, 70], dtype=dtype, causal=causal, window=window)
    run([40, 200], [90, 130], dtype=dtype, causal=causal, window=window)


@BOTH
@pytest.mark.parametrize("window", [0, 20])
def test_prefixes(window, dtype):
    run([200, 64, 33, 1], dtype=dtype, prefix=[70, 0, 33, 1], window=window)
    run([300], dtype=dtype, prefix=[65], window=window, heads=1)
    # beyond the keys, and below 0: as all of them, none
    q, k, v = inputs([50], [50], 2, 1, 64, dtype, False, 3)
    far = L.attention(q, k, v, prefix=torch.tensor([999], dtype=torch.int32).cuda(), window=window)
    full = L.attention(q, k, v, causal=False)
    assert torch.equal(far.out, full.out)
    none = L.attention(q, k, v, prefix=torch.tensor([-5], dtype=torch.int32).cuda(), window=window)
    assert torch.equal(none.out, L.attention(q, k, v, window=window).out)


@BOTH
def test_lengths_of_keys(dtype):
    # fewer keys than queries: the first queries see nothing
    got, grads = run([100, 7, 40], [30, 0, 200], dtype=dtype, heads=4, kv=2)
    assert (got.out[:70] == 0).all() and (got.lse[:, :70] == -math.inf).all()
    assert (got.out[100:107] == 0).all() and (grads.dq[:70] == 0).all()
    # keys that no query sees
    got, grads = run([5, 0], [100, 20], dtype=dtype, window=10)
    assert (grads.dk[:80] == 0).all() and (grads.dv[100:] == 0).all()
    run([1, 1, 1], [300, 17, 1], dtype=dtype, causal=False)


@BOTH
@pytest.mark.parametrize("softcap,slopes", [(20.0, False), (0.0, True), (2.0, True)])
def test_shaped_scores(softcap, slopes, dtype):
    run([140, 65], dtype=dtype, softcap=softcap, slopes=slopes, heads=4, kv=2, dim=128)
    run([80], [120], dtype=dtype, softcap=softcap, slopes=slopes, causal=False, dim=72)
    run([80, 90], dtype=dtype, softcap=softcap, slopes=slopes, prefix=[30, 90], window=9)


@BOTH
def test_large_and_small_scores(dtype):
    run([130], dtype=dtype, scale=2.0, heads=1)       # scores to about 60: one key takes all
    run([130], dtype=dtype, scale=-0.3, heads=1)
    run([130], dtype=dtype, scale=0.0, heads=1)


def test_many_rows():
    run([1500, 700], heads=4, kv=2, dim=128)
    run([2100], heads=2, kv=1, dim=64, window=300)


@BOTH
@pytest.mark.parametrize("shape", [dict(), dict(window=100), dict(prefix=[900, 5]),
                                   dict(softcap=10.0, slopes=True), dict(causal=False)])
def test_parts(shape, dtype):
    """Few tiles of queries or keys: keys and queries in parts."""
    run([700, 900], dtype=dtype, heads=1, dim=64, **shape)
    run([3, 600], [1500, 1100], dtype=dtype, heads=2, dim=80, **shape)
    run([900, 1200], [40, 1], dtype=dtype, heads=4, dim=128, **{**shape, "prefix": None})
    run([1, 1], [2000, 1300], dtype=dtype, heads=4, **{**shape, "prefix": None})


@BOTH
def test_batches(dtype):
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(3, n, h, 64, generator=g).to(dtype).cuda()
               for n, h in ((40, 4), (75, 2), (75, 2)))
    got = L.attention(q, k, v)
    flat = [t.reshape(-1, *t.shape[2:]) for t in (q, k, v)]
    off = dict(q_begin=offsets([40] * 3).cuda(), k_begin=offsets([75] * 3).cuda())
    want = L.attention(*flat, **off)
    assert torch.equal(got.out.view(120, 4, 64), want.out) and torch.equal(got.lse, want.lse)
    dout = torch.randn(q.shape, generator=g).to(dtype).cuda()
    a = L.attention_backward(dout, q, k, v, got.out, got.lse)
    b = L.attention_backward(dout.view(120, 4, 64), *flat, want.out, want.lse, **off)
    assert all(torch.equal(x.reshape(y.shape), y) for x, y in zip(a, b))


@pytest.mark.parametrize("first,behind", [(9, 50), (128, 0), (301, 300)])
def test_rows_outside_are_left(first, behind):
    lens = [40, 30]
    q, k, v = inputs(lens, lens, 2, 1, 64, torch.bfloat16, True, 4, first, behind)
    for t in (q, k, v):                               # nothing of these is used
        t[:first] = math.nan
        t[first + 70:] = math.inf
    qb = offsets(lens, first).cuda()
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    got = L.attention(q, k, v, q_begin=qb, out=out)
    inner = slice(first, first + 70)
    want = L.attention(q[inner], k[inner], v[inner], q_begin=offsets(lens).cuda())
    assert torch.equal(out[inner], want.out) and torch.equal(got.lse[:, inner], want.lse)
    assert (out[:first] == 7).all() and (out[first + 70:] == 7).all()
    dout = torch.randn(q.shape, device="cuda").bfloat16()
    dqkv = torch.full((q.shape[0], 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    L.attention_backward(dout, q, k, v, out, got.lse, q_begin=qb, dq=dqkv[:, :2], dk=dqkv[:, 2:3],
                         dv=dqkv[:, 3:])
    back = L.attention_backward(dout[inner], q[inner], k[inner], v[inner], want.out, want.lse,
                                q_begin=offsets(lens).cuda())
    # Not bit by bit: sums are cut into parts by the buffers' rows (671 x 2 heads / 256: two parts of
    # the queries; of 70 one), so that binary32 additions come in another order.  Both are held to
    # the formula, with the bounds of their roundings, which no order of the additions leaves.
    lse = got.lse[:, inner].cpu().double()
    want, err = R.attention(*(t[inner].cpu().double() for t in (q, k, v)), offsets(lens), offsets(lens),
                            64 ** -0.5, dtype=torch.bfloat16, dout=dout[inner].cpu().double(),
                            out=out[inner].cpu().double(), lse=lse)
    for n, whole in (("dq", dqkv[inner, :2]), ("dk", dqkv[inner, 2:3]), ("dv", dqkv[inner, 3:])):
        R.close(whole, want[n], err[n], f"{n} of the rows between, {first} before")
        R.close(getattr(back, n), want[n], err[n], f"{n} of the rows alone")
    assert (dqkv[:first] == 5).all() and (dqkv[first + 70:] == 5).all()


def test_not_finite_stays_in_its_sequence():
    q, k, v = inputs([40, 40, 40], [40, 40, 40], 2, 1, 64, torch.bfloat16, False, 5)
    how = dict(q_begin=offsets([40, 40, 40]).cuda())
    clean = L.attention(q, k, v, **how)
    k[45], v[50], q[60] = math.inf, math.nan, math.nan
    got = L.attention(q, k, v, **how)
    for s in (slice(0, 40), slice(80, 120)):
        assert torch.equal(got.out[s], clean.out[s]) and torch.equal(got.lse[:, s], clean.lse[:, s])
    assert got.out[60].isnan().all() and got.lse[:, 60].isnan().all()


@pytest.mark.parametrize("dtype", [torch.float32])
def test_gradient_by_differences(dtype):
    """Of a smooth function of the outputs, along random directions, in binary32: differences of
    the 64-bit form of the forward pass."""
    lens, heads, kv, dim = [23, 40], 4, 2, 24
    q, k, v = inputs(lens, lens, heads, kv, dim, dtype, False, 6)
    qb = offsets(lens)
    sl = torch.rand(heads) * 0.2
    how = dict(causal=True, window=30, softcap=5.0)
    pre = torch.tensor([4, 9], dtype=torch.int32)
    got = L.attention(q, k, v, q_begin=qb.cuda(), prefix=pre.cuda(), slopes=sl.cuda(), **how)
    w = torch.randn(q.shape, generator=torch.Generator().manual_seed(1))
    grads = L.attention_backward(w.cuda(), q, k, v, got.out, got.lse, q_begin=qb.cuda(),
                                 prefix=pre.cuda(), slopes=sl.cuda(), **how)

    def loss(*t):
        r, _ = R.attention(*t, qb, qb, dim ** -0.5, prefix=pre, slopes=sl, dtype=dtype, **how)
        return float((r["out"] * w.double()).sum())

    base = [t.cpu().double() for t in (q, k, v)]
    for i, g in enumerate(grads):
        step = torch.randn(base[i].shape, generator=torch.Generator().manual_seed(10 + i)).double()
        at = lambda e: loss(*[t + e * step if j == i else t for j, t in enumerate(base)])  # noqa: E731
        h = 1e-4
        want = (8 * (at(h) - at(-h)) - (at(2 * h) - at(-2 * h))) / (12 * h)
        have = float((g.cpu().double() * step).sum())
        # the difference's error is of h^4 and of 1e-16 / h; the gradient's are binary32 ones of
        # sums of up to 100 terms
        assert abs(have - want) <= 1e-5 * float((g.cpu().double() * step).abs().sum())


def test_equal_bits_streams_and_graphs():
    q, k, v = inputs([200, 100], [200, 100], 4, 2, 64, torch.bfloat16, True, 8)
    how = dict(q_begin=offsets([200, 100]).cuda())
    dout = torch.randn(q.shape, device="cuda").bfloat16()
    one = L.attention(q, k, v, **how)
    grads = L.attention_backward(dout, q, k, v, one.out, one.lse, **how)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        two = L.attention(q, k, v, **how)
        again = L.attention_backward(dout, q, k, v, two.out, two.lse, **how)
    s.synchronize()
    assert torch.equal(one.out, two.out) and torch.equal(one.lse, two.lse)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = L.attention(q, k, v, **how)
        kept_grads = L.attention_backward(dout, q, k, v, kept.out, kept.lse, **how)
    for turn in range(3):
        q.copy_(torch.randn(q.shape, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        one = L.attention(q, k, v, **how)
        grads = L.attention_backward(dout, q, k, v, one.out, one.lse, **how)
        torch.cuda.synchronize()
        assert torch.equal(one.out, kept.out)
        assert all(torch.equal(a, b) for a, b in zip(grads, kept_grads))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("how", [dict(softcap=1e-39), dict(softcap=1e-39, scale=1e30), dict(scale=3e38)])
def test_factors_beyond_binary32(how, dtype):
    """Sums of products that are 0 have scores of 0 whatever they are multiplied by."""
    _, k, v = inputs([70], [70], 2, 1, 64, dtype, False, 10)
    q = torch.zeros(70, 2, 64, dtype=dtype, device="cuda")
    got = L.attention(q, k, v, causal=False, **how)
    ones = L.attention(q, k, v, causal=False)
    assert torch.equal(got.out, ones.out) and torch.equal(got.lse, ones.lse)
    dout = torch.ones_like(q)
    back = L.attention_backward(dout, q, k, v, got.out, got.lse, causal=False, **how)
    # every score's weight is 1 / 70, of the sum of whose roundings, half a step of dtype and a
    # few of binary32 each, there are 2 x 70
    want = 2.0
    assert (back.dv.double() - want).abs().max() <= want * (torch.finfo(dtype).eps + 1e-5)


def test_nothing_to_do():
    e = torch.empty(0, 2, 64, device="cuda")
    assert L.attention(e, e, e).out.shape == (0, 2, 64)
    q = torch.randn(5, 2, 64, device="cuda")
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 3.0)
    L.attention(q, q, q, q_begin=none, out=out)
    assert (out == 3).all()
    # no keys at all
    got = L.attention(q, e, e)
    assert (got.out == 0).all() and (got.lse == -math.inf).all()
    grads = L.attention_backward(q, q, e, e, got.out, got.lse)
    assert (grads.dq == 0).all() and grads.dk.shape == (0, 2, 64)
    # no queries
    grads = L.attention_backward(e, e, q, q, e, torch.empty(2, 0, device="cuda"))
    assert (grads.dk == 0).all() and (grads.dv == 0).all()


def test_offsets_beyond_the_rows_are_cut():
    q, k, v = inputs([40], [40], 1, 1, 64, torch.bfloat16, False, 9)
    wild = torch.tensor([-3, 20, 2000], dtype=torch.int32).cuda()
    got = L.attention(q, k, v, q_begin=wild)
    want = L.attention(q, k, v, q_begin=offsets([20, 20]).cuda())
    assert torch.equal(got.out, want.out)
