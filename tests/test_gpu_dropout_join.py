"""GPU checks of dropout and the block join, forward and backward, against
plain 64-bit forms.

Bounds, derived before any run.  An output is off by half a step of its type
relative to its value, plus binary32 roundings of what is added up for it, of
2^-24 relative each.  A row's sums add at most 16 values in a lane, 6 levels
across a wave and 16 waves: under 40 roundings, halved by the square root, so
that K_ROW = 48 covers statistics, products and the norm's formula; second
norms see the first one's errors too: twice that.  Sums over rows take one
rounding for each row besides."""
import numpy as np
import pytest
import torch

import train_ref as R
from gpu_util import DEV, say
from weight_communication_compression_amd import lowbit as L

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f32": torch.float32}
K_ROW = 48


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    L.lib()
    yield
    torch.cuda.synchronize()


def normal(g, shape, dtype, std=1.0, mean=0.0):
    return torch.from_numpy((g.standard_normal(shape) * std + mean).astype(np.float32)).to(T[dtype])


# --------------------------------------------------------------- dropout ---
def want_dropout(x, r, p, seed, offset=0):
    """Bit for bit: one product and one sum in binary32, rounded once."""
    cut, factor = R.cut_and_factor(p)
    keep = R.draws(offset, x.numel(), seed) >= cut
    y = torch.where(torch.from_numpy(keep), x.float() * np.float32(factor), torch.zeros(()))
    return (y if r is None else r.float() + y).to(x.dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0 - 2.0 ** -16, 1.0])
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 511, 1024, 1025, 2048 * 5 + 13])
def test_dropout(n, p, dtype):
    say("dropout", n, p, dtype)
    g = np.random.default_rng(n)
    x, r = normal(g, n, dtype), normal(g, n, dtype)
    seed = 0x1234567890ABCDEF + n
    for res in (None, r):
        y = L.dropout(x.to(DEV), p, seed, residual=None if res is None else res.to(DEV))
        assert torch.equal(y.cpu(), want_dropout(x, res, p, seed))
    dx = L.dropout_backward(x.to(DEV), p, seed)
    assert torch.equal(dx.cpu(), want_dropout(x, None, p, seed))


def test_dropout_pieces_draw_the_whole_mask():
    g = np.random.default_rng(3)
    x = normal(g, 40000, "f32")
    whole = L.dropout(x.to(DEV), 0.3, 5).cpu()
    for cut in (8, 2048, 2056, 39992):
        parts = [L.dropout(x[:cut].to(DEV), 0.3, 5),
                 L.dropout(x[cut:].to(DEV), 0.3, 5, index_offset=cut)]
        assert torch.equal(torch.cat(parts).cpu(), whole)


@pytest.mark.parametrize("offset", [2 ** 33 - 1024, 2 ** 33 - 8, 2 ** 33, 2 ** 40 + 8])
def test_dropout_far_offsets(offset):
    """Pair indices that pass 32 bits inside a tile."""
    g = np.random.default_rng(4)
    x = normal(g, 5000, "bf16")
    y = L.dropout(x.to(DEV), 0.4, 77, index_offset=offset)
    assert torch.equal(y.cpu(), want_dropout(x, None, 0.4, 77, offset))


def test_dropout_drops_nan_and_infinity():
    x = torch.full((4096,), float("nan"))
    x[1::2] = float("inf")
    y = L.dropout(x.to(DEV), 0.5, 1).cpu()
    dropped = torch.from_numpy(R.draws(0, 4096, 1) < 32768)
    assert torch.equal(y[dropped], torch.zeros(int(dropped.sum())))
    assert not torch.isfinite(y[~dropped]).any()


def test_dropout_in_place_and_streams():
    g = np.random.default_rng(6)
    x, r = normal(g, 12345, "bf16"), normal(g, 12345, "bf16")
    want = want_dropout(x, r, 0.2, 9)
    a, b = x.to(DEV), r.to(DEV)
    assert L.dropout(a, 0.2, 9, residual=b, out=b) is b and torch.equal(b.cpu(), want)
    b = r.to(DEV)
    assert L.dropout(a, 0.2, 9, residual=b, out=a) is a and torch.equal(a.cpu(), want)
    side = torch.cuda.Stream()
    a = x.to(DEV)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = L.dropout(a, 0.2, 9)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y.cpu(), want_dropout(x, None, 0.2, 9))


def test_dropout_beyond_31_bits():
    n = 2 ** 31 + 4099
    x = torch.ones(n, dtype=torch.bfloat16, device=DEV)
    y = L.dropout(x, 0.25, 11)
    at = n - 8192 - n % 8
    keep = torch.from_numpy(R.draws(at, n - at, 11) >= 16384)
    want = torch.where(keep, torch.tensor(65536 / 49152), torch.zeros(())).to(torch.bfloat16)
    assert torch.equal(y[at:].cpu(), want)


# ------------------------------------------------------------------ join ---
CASES = [  # rows, cols, block, stream, params, norm, group (0: no gate), biases, p, a, given
    (1, 1, "f32", "f32", "f32", "rms", 1, True, 0.0, 1.0, True),
    (3, 7, "bf16", "bf16", "bf16", "layer", 2, True, 0.0, 1.0, True),
    (5, 64, "bf16", "f32", "f32", "rms", 5, False, 0.1, 0.5, True),
    (9, 513, "bf16", "bf16", "bf16", "layer", 1, True, 0.3, 1.0, True),
    (4, 1024, "f32", "f32", "f32", "layer", 0, False, 0.0, 1.0, False),
    (33, 1155, "bf16", "f32", "f32", "layer", 7, True, 0.2, 0.7, True),
    (17, 2048, "bf16", "bf16", "f32", "rms", 17, True, 0.0, 1.0, True),
    (6, 4096, "bf16", "bf16", "bf16", "rms", 4, False, 0.1, 1.0, True),
    (5, 4104, "bf16", "f32", "bf16", "layer", 3, True, 0.1, -1.0, True),
    (3, 8191, "f32", "f32", "f32", "rms", 2, True, 0.5, 1.0, True),
    (2, 16384, "bf16", "f32", "bf16", "layer", 2, True, 0.1, 1.0, True),
    (2, 16001, "f32", "f32", "f32", "layer", 1, True, 0.1, 1.0, True),
    # more rows than workgroups: several rows each, groups within and across them
    (8200, 40, "bf16", "bf16", "bf16", "rms", 7, True, 0.1, 1.0, True),
    (4500, 520, "bf16", "bf16", "bf16", "layer", 2048, True, 0.0, 1.0, True),
    (2100, 2056, "bf16", "bf16", "bf16", "rms", 1, False, 0.1, 1.0, True),
]


def make_join(rows, cols, bt, st, pt, norm, group, biases, p, a, given, seed=0):
    g = np.random.default_rng(rows * 7919 + cols + seed)
    loud = np.where(g.random(cols) < 0.02, 20.0, 1.0)
    s = {"f": normal(g, (rows, cols), "f32", 0.5, 0.3) * torch.from_numpy(loud).float(),
         "x": normal(g, (rows, cols), "f32") * torch.from_numpy(loud).float()}
    s["f"], s["x"] = s["f"].to(T[bt]), s["x"].to(T[st])
    s["post_weight"] = normal(g, cols, pt, 0.1, 1.0) if given else None
    s["pre_weight"] = normal(g, cols, pt, 0.1, 1.0) if given else None
    s["post_bias"] = normal(g, cols, pt, 0.1) if biases else None
    s["pre_bias"] = normal(g, cols, pt, 0.1) if biases else None
    s["gate"] = normal(g, (-(-rows // group), cols), pt, 0.3, 0.5) if group else None
    how = dict(rows_per_gate=group, norm=norm, residual_scale=a, eps=1e-5, p=p,
               seed=0xFEDCBA9876543210 + seed)
    s["dx_out"] = normal(g, (rows, cols), st, 1e-2)
    s["dz"] = normal(g, (rows, cols), bt, 1e-2)
    return s, how


NAMES = ("post_weight", "post_bias", "gate", "pre_weight", "pre_bias")


def gpu(t):
    return None if t is None else t.to(DEV)


def opt64(t):
    return None if t is None else R.f64(t)


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_join_and_backward(case):
    say("join", case)
    rows, cols, bt, st = case[:4]
    s, how = make_join(*case)
    params = {k: gpu(s[k]) for k in NAMES}
    out = L.block_join(gpu(s["f"]), gpu(s["x"]), **params, **how)
    p64 = {k: opt64(s[k]) for k in NAMES}
    y, z, stats, size = R.join(R.f64(s["f"]), R.f64(s["x"]), p64["post_weight"],
                               p64["post_bias"], p64["gate"], how["rows_per_gate"],
                               p64["pre_weight"], p64["pre_bias"], how["norm"],
                               how["residual_scale"], 1e-5, how["p"], how["seed"])
    say("  forward ran")
    R.within(R.f64(out.x_out), y, R.half_step(T[st]) * np.abs(y) + K_ROW * R.U * size, "x_out")
    w = 1.0 if p64["pre_weight"] is None else np.abs(p64["pre_weight"])
    r2 = stats[:, 3:]
    zsize = np.abs(z) + w * r2 * (size + size.mean(1, keepdims=True) + np.abs(y))
    R.within(R.f64(out.z), z, R.half_step(T[bt]) * np.abs(z) + 2 * K_ROW * R.U * zsize, "z")
    f = np.abs(R.f64(s["f"])).mean(1)
    # a centred sum's error counts against the spread: (values / spread)^2 at most
    bound = K_ROW * R.U * np.stack([f, stats[:, 1] * (1 + f * stats[:, 1]),
                                    size.mean(1), r2[:, 0] * (1 + 2 * size.mean(1) * r2[:, 0])], 1)
    R.within(R.f64(out.stats), stats, 2 * bound, "stats")

    back = L.block_join_backward(gpu(s["dx_out"]), gpu(s["dz"]), gpu(s["f"]), out.x_out,
                                 out.stats, **params, **how)
    want = R.join_back(R.f64(s["dx_out"]), R.f64(s["dz"]), R.f64(s["f"]), R.f64(out.x_out),
                       R.f64(out.stats), p64["post_weight"], p64["post_bias"], p64["gate"],
                       how["rows_per_gate"], p64["pre_weight"], how["norm"],
                       how["residual_scale"], how["p"], how["seed"])
    say("  backward ran")
    for name, got in back._asdict().items():
        if got is None:
            assert s[name[1:]] is None
            continue
        v, size = want[name]
        over_rows = 0 if name in ("df", "dx") else rows
        R.within(R.f64(got).reshape(v.shape), v, R.half_step(got.dtype) * np.abs(v)
                 + (2 * K_ROW + over_rows) * R.U * size, name)


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_join_gradient_against_differences(norm):
    """The formulas themselves: central differences of the 64-bit forward."""
    s, how = make_join(4, 24, "f32", "f32", "f32", norm, 3, True, 0.25, 0.8, True, seed=5)
    out = L.block_join(gpu(s["f"]), gpu(s["x"]), **{k: gpu(s[k]) for k in NAMES}, **how)
    got = L.block_join_backward(gpu(s["dx_out"]), gpu(s["dz"]), gpu(s["f"]), out.x_out, out.stats,
                                **{k: gpu(s[k]) for k in NAMES}, **how)._asdict()
    v = {k: R.f64(s[k]) for k in ("f", "x") + NAMES}
    dxo, dz = R.f64(s["dx_out"]), R.f64(s["dz"])

    def loss():
        y, z, _, _ = R.join(v["f"], v["x"], v["post_weight"], v["post_bias"], v["gate"],
                            how["rows_per_gate"], v["pre_weight"], v["pre_bias"], norm,
                            how["residual_scale"], how["eps"], how["p"], how["seed"])
        return (y * dxo).sum() + (z * dz).sum()

    for name, a in v.items():
        grad = R.f64(got["d" + name]).reshape(-1)
        flat = a.reshape(-1)
        for i in range(0, flat.size, max(1, flat.size // 24)):
            old, h = flat[i], 1e-5
            flat[i] = old + h
            up = loss()
            flat[i] = old - h
            down = loss()
            flat[i] = old
            assert abs((up - down) / (2 * h) - grad[i]) <= 2e-6, (name, i)


def test_join_in_place_equal_bits_and_graph():
    """In place, twice, on another stream and replayed from a graph: equal bits."""
    case = (700, 1032, "bf16", "bf16", "bf16", "rms", 100, True, 0.1, 1.0, True)
    s, how = make_join(*case)
    params = {k: gpu(s[k]) for k in NAMES}
    f, x, dxo, dz = (gpu(s[k]) for k in ("f", "x", "dx_out", "dz"))
    out = L.block_join(f, x, **params, **how)
    ref = L.block_join_backward(dxo, dz, f, out.x_out, out.stats, **params, **how)
    f2, x2 = f.clone(), x.clone()
    again = L.block_join(f2, x2, x_out=x2, z=f2, **params, **how)
    assert torch.equal(x2, out.x_out) and torch.equal(f2, out.z) and again.x_out is x2
    dxo2, dz2 = dxo.clone(), dz.clone()
    back = L.block_join_backward(dxo2, dz2, f, out.x_out, out.stats, dx=dxo2, df=dz2, **params, **how)
    for a, b in zip(back, ref):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        L.block_join_backward(dxo, dz, f, out.x_out, out.stats, **params, **how)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fwd = L.block_join(f, x, **params, **how)
        bwd = L.block_join_backward(dxo, dz, f, fwd.x_out, fwd.stats, **params, **how)
    for k in range(3):
        for t in (*fwd, *bwd):
            t.fill_(float("nan"))
        torch.ones(1000, device=DEV).sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((*fwd, *bwd), (*out, *ref)):
            assert torch.equal(a, b), k


def test_join_rows_of_nothing_and_of_nan():
    """A row of zeros with eps = 0 and a row with a NaN spoil themselves alone;
    p = 1 leaves the residual alone whatever f holds."""
    s, how = make_join(6, 264, "bf16", "f32", "f32", "rms", 6, True, 0.0, 1.0, True)
    params = {k: gpu(s[k]) for k in NAMES}
    clean = L.block_join(gpu(s["f"]), gpu(s["x"]), **params, **how)
    f = s["f"].clone()
    f[2, 17] = float("nan")
    out = L.block_join(gpu(f), gpu(s["x"]), **params, **how)
    assert torch.isnan(out.x_out[2]).all() and torch.isnan(out.z[2]).all()
    for r in (0, 1, 3, 4, 5):
        assert torch.equal(out.x_out[r], clean.x_out[r]) and torch.equal(out.z[r], clean.z[r])
    how["p"] = 1.0
    f[:] = float("inf")
    out = L.block_join(gpu(f), gpu(s["x"]), **params, **how)
    assert torch.equal(out.x_out.cpu(), s["x"]) and torch.isfinite(out.z).all()


def test_join_no_rows():
    for norm in ("rms", "layer"):
        f = torch.empty(0, 64, device=DEV)
        w = torch.ones(64, device=DEV)
        out = L.block_join(f, f, post_weight=w, norm=norm)
        assert out.x_out.shape == (0, 64) and out.stats.shape == (0, 4)
        g = L.block_join_backward(f, f, f, f, out.stats, post_weight=w, pre_bias=w, norm=norm)
        assert torch.equal(g.dpost_weight, torch.zeros_like(w))
        assert torch.equal(g.dpre_bias, torch.zeros_like(w)) and g.dgate is None
