"""Host-side checks of rotary, attention and orthogonalize (no GPU needed): refusals before any
HIP call, workspace sizes, frequencies, what the binding passes on, and the plain forms that the
GPU tests compare with."""
import ctypes
import math

import numpy as np
import pytest
import torch

import block_ref as R
from weight_communication_compression_amd import lowbit as L

OK16 = ctypes.c_void_p(0x1000)          # never read: every call here is refused
OFF = ctypes.c_void_p(0x1008)
OFF1 = ctypes.c_void_p(0x1001)


# ------------------------------------------------------------------ rotary --
def _rotary(x=OK16, freqs=OK16, positions=OK16, y=OK16, back=False, **change):
    v = dict(rows=10, rows_per_sequence=0, heads=4, head_dim=64, rot_dim=32, layout=0, type=0,
             scale=1.0, x=(256, 64), y=(256, 64))
    if y is OK16 and x is OK16:
        y = ctypes.c_void_p(0x100000)
    v.update(change if "y_strides" not in change else {k: w for k, w in change.items() if k != "y_strides"})
    ys = change.get("y_strides", v["y"])
    p = L.RotaryParams(v["rows"], v["rows_per_sequence"], *v["x"], *ys, v["heads"], v["head_dim"],
                       v["rot_dim"], v["layout"], v["type"], v["scale"])
    call = L.lib().lowbit_rotary_backward if back else L.lib().lowbit_rotary
    return call(x, freqs, positions, p, y, None)


@pytest.mark.parametrize("back", [False, True])
def test_rotary_refusals(back):
    for bad in (dict(rows=-1), dict(rows=1 << 31), dict(heads=0), dict(heads=65537),
                dict(head_dim=1), dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=66),
                dict(layout=2), dict(layout=-1), dict(type=2), dict(scale=math.inf),
                dict(scale=math.nan), dict(positions=None), dict(freqs=None),
                dict(freqs=ctypes.c_void_p(0x1004)), dict(positions=ctypes.c_void_p(0x1004)),
                # two elements of y would share a place
                dict(y_strides=(255, 64)), dict(y_strides=(256, 63)), dict(y_strides=(0, 64)),
                dict(y_strides=(256, 0)), dict(y_strides=(64, 639)), dict(y_strides=(-256, 64)),
                dict(y_strides=(1 << 41, 64))):
        assert _rotary(back=back, **bad) == L.EINVAL, bad
    assert _rotary(back=back, rows=0, y_strides=(1, 64)) == L.OK
    call = L.lib().lowbit_rotary
    assert call(OK16, OK16, OK16, None, OK16, None) == L.EINVAL
    p = L.RotaryParams(10, 0, 256, 64, 256, 64, 4, 64, 32, 0, 0, 1.0)
    assert call(None, OK16, OK16, p, OK16, None) == L.EINVAL
    assert call(OK16, OK16, OK16, p, None, None) == L.EINVAL
    assert call(ctypes.c_void_p(0x1002), OK16, OK16, p, OK16, None) == L.EINVAL
    # in place with other strides
    p.x_row = 512
    assert call(OK16, OK16, OK16, p, OK16, None) == L.EINVAL


def test_frequencies():
    for rot, base in ((2, 10000.0), (64, 10000.0), (128, 5e5)):
        plain, scale = L.rotary_frequencies(rot, base)
        want = base ** (-2.0 * np.arange(rot // 2) / rot)
        assert scale == 1.0 and np.allclose(plain, want, rtol=1e-14)
        lin, _ = L.rotary_frequencies(rot, base, "linear", 4.0)
        assert np.allclose(lin, want / 4, rtol=1e-14)
        big, _ = L.rotary_frequencies(rot, base, "base", 4.0)
        assert big[0] == 1.0 and (rot == 2 or np.isclose(big[-1], want[-1] / 4, rtol=1e-12))
        parts, scale = L.rotary_frequencies(rot, base, "parts", 4.0, original_length=4096)
        assert np.isclose(scale, 0.1 * math.log(4.0) + 1)
        turns = 4096 * want / (2 * math.pi)
        assert np.allclose(parts.numpy()[turns >= 32], want[turns >= 32])
        assert np.allclose(parts.numpy()[turns <= 1], want[turns <= 1] / 4)
        assert ((parts.numpy() <= want * (1 + 1e-14)) & (parts.numpy() >= want / 4 * (1 - 1e-14))).all()


def test_frequency_refusals():
    for bad in (dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=1 << 20), dict(base=0.0),
                dict(base=-1.0), dict(base=math.inf), dict(scaling="other"), dict(factor=0.0),
                dict(scaling="linear", factor=math.nan),
                dict(scaling="parts", factor=0.5, original_length=10), dict(scaling="parts"),
                dict(scaling="parts", original_length=10, slow_turns=5.0, fast_turns=5.0),
                dict(scaling="parts", original_length=10, slow_turns=-1.0)):
        with pytest.raises(L.LowbitError):
            L.rotary_frequencies(**{"rot_dim": 8, **bad})


def test_rotary_binding_refusals():
    x, f = torch.zeros(4, 2, 8), torch.zeros(4, dtype=torch.float64)
    at = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: L.rotary(x, f, at),                       # of the host
                 lambda: L.rotary(x[0, 0], f, at[:1]), lambda: L.rotary(x, f.float(), at),
                 lambda: L.rotary(x, f, at[:3]), lambda: L.rotary(x, f, at.int()),
                 lambda: L.rotary(x, f, at, layout="other"), lambda: L.rotary(x[..., ::2], f, at),
                 lambda: L.rotary(x, f, at, out=x[:3]), lambda: L.rotary(x, f, at, out=x.half()),
                 lambda: L.rotary(x.half(), f, at),
                 lambda: L.rotary(torch.zeros(4, 3, 2, 8).transpose(0, 1)[:, :2], f)):
        with pytest.raises(L.LowbitError):
            call()


# --------------------------------------------------------------- attention --
NAMES = ("q", "k", "v", "out", "dout", "dq", "dk", "dv")


def _params(**change):
    v = dict(q_rows=100, k_rows=100, window=0, sequences=2, q_heads=4, kv_heads=2, head_dim=64,
             type=1, causal=1, scale=0.125, softcap=0.0)
    strides = {n: (64 * (2 if n[-1] in "kv" else 4), 64) for n in NAMES}
    for k, w in change.items():
        (strides if k in NAMES else v)[k] = w
    return L.AttentionParams(*v.values(), *[s for n in NAMES for s in strides[n]])


def _both(p, q=OK16, k=OK16, v=OK16, qb=OK16, kb=None, pre=None, sl=None, out=OK16, lse=OK16,
          ws=OK16, bytes=1 << 40, dq=OK16, dk=OK16, dv=OK16, dout=OK16):
    lib = L.lib()
    return (lib.lowbit_attention(q, k, v, qb, kb, pre, sl, p, out, lse, ws, bytes, None),
            lib.lowbit_attention_backward(dout, q, k, v, out, lse, qb, kb, pre, sl, p, dq, dk, dv,
                                          ws, bytes, None))


def test_attention_refusals():
    for bad in (dict(q_rows=-1), dict(q_rows=(1 << 29) + 1), dict(k_rows=-1),
                dict(k_rows=(1 << 29) + 1), dict(window=-1), dict(sequences=-1),
                dict(sequences=(1 << 24) + 1), dict(q_heads=0), dict(q_heads=4097),
                dict(kv_heads=0), dict(kv_heads=3), dict(kv_heads=8), dict(head_dim=0),
                dict(head_dim=4), dict(head_dim=63), dict(type=2), dict(causal=2),
                dict(scale=math.inf), dict(scale=math.nan), dict(softcap=-1.0),
                dict(softcap=math.nan), dict(q=(56, 64)), dict(q=(1 << 23, 64)), dict(k=(129, 64)),
                dict(v=(128, 63)), dict(v=(128, -64)), dict(out=(128, 64)), dict(out=(256, 56)),
                dict(out=(256, 0)), dict(k_rows=101)):
        p = _params(**bad)
        assert _both(p) == (L.EINVAL, L.EINVAL) or ("out" in bad and _both(p)[0] == L.EINVAL), bad
    for bad in (dict(dq=(128, 64)), dict(dk=(64, 64)), dict(dv=(128, 0)), dict(dout=(60, 64)),
                dict(dk=(1 << 23, 64))):
        assert _both(_params(**bad))[1] == L.EINVAL, bad
    assert _both(_params(head_dim=136, **{n: (1088, 136) for n in NAMES})) == \
        (L.EUNSUPPORTED, L.EUNSUPPORTED)
    ok = _params()
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(q=OFF), dict(k=OFF), dict(v=OFF),
                dict(out=None), dict(out=OFF), dict(lse=None), dict(lse=OFF), dict(qb=OFF1),
                dict(kb=OFF1), dict(pre=OFF1), dict(sl=OFF1)):
        assert _both(ok, **bad) == (L.EINVAL, L.EINVAL), bad
    for bad in (dict(ws=None), dict(ws=OFF), dict(bytes=100 * 4 * 8 - 1), dict(dq=None),
                dict(dk=OFF), dict(dv=None), dict(dout=OFF)):
        assert _both(ok, **bad)[1] == L.EINVAL, bad
    # equal sequences have to divide the rows
    assert _both(_params(sequences=3), qb=None) == (L.EINVAL, L.EINVAL)
    assert _both(_params(sequences=3, q_rows=99), qb=None) == (L.EINVAL, L.EINVAL)
    assert _both(_params(k_rows=101), qb=OK16, kb=None) == (L.EINVAL, L.EINVAL)
    assert _both(None) == (L.EINVAL, L.EINVAL)
    # nothing to do
    assert _both(_params(sequences=0)) == (L.OK, L.OK)
    assert _both(_params(q_rows=0, k_rows=0)) == (L.OK, L.OK)


def test_attention_workspace():
    ws = L.lib().lowbit_attention_workspace
    assert ws(_params(), 1) >= 100 * 4 * 8 and ws(_params(q_rows=0, k_rows=0), 1) == 0
    assert ws(_params(), 0) == 0 and ws(_params(q_rows=0, k_rows=0), 0) == 0
    # few queries against many keys, and the other way round: parts of sums
    few = _params(q_rows=2, k_rows=20000)
    assert ws(few, 0) > 0 and _both(few, kb=OK16, bytes=ws(few, 0) - 1)[0] == L.EINVAL
    assert _both(few, kb=OK16, ws=None)[0] == L.EINVAL
    many = _params(q_rows=20000, k_rows=2)
    assert ws(many, 0) == 0 and ws(many, 1) > 20000 * 4 * 8
    for back in (0, 1):
        assert ws(_params(type=3), back) == -1 and ws(_params(head_dim=136), back) == -1
        assert ws(None, back) == -1


def test_attention_binding_refusals():
    q, k = torch.zeros(10, 4, 16), torch.zeros(10, 2, 16)
    b = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: L.attention(q, k, k),                     # of the host
                 lambda: L.attention(q, k, k[:9]), lambda: L.attention(q, k.bfloat16(), k),
                 lambda: L.attention(q, k[..., :8], k[..., :8]), lambda: L.attention(q[0], k[0], k[0]),
                 lambda: L.attention(k, q, q), lambda: L.attention(q, k[:, :0], k[:, :0]),
                 lambda: L.attention(q, k, k, q_begin=b.long()),
                 lambda: L.attention(q, k, k, q_begin=b, k_begin=b[:2]),
                 lambda: L.attention(q[None], k[None], k[None], q_begin=b),
                 lambda: L.attention(q[None], k[None].repeat(2, 1, 1, 1), k[None].repeat(2, 1, 1, 1)),
                 lambda: L.attention(q, k, k, prefix=b), lambda: L.attention(q, k, k, slopes=b.float()),
                 lambda: L.attention(q, k, k, out=k), lambda: L.attention(q.half(), k.half(), k.half()),
                 lambda: L.attention_backward(q, q, k, k, q, torch.zeros(3, 10))):
        with pytest.raises(L.LowbitError):
            call()


def test_strides_that_the_binding_passes_on():
    t = torch.zeros(6, 7, 16)
    assert [L._heads(v, "t") for v in (t, t[:, 2:5], t[:1], t[:, :1])] \
        == [(6, 112, 16), (6, 112, 16), (1, 112, 16), (6, 112, 16)]
    four = torch.zeros(2, 3, 5, 8)
    assert L._heads(four[:, :, 1:3], "t") == (6, 40, 8)
    with pytest.raises(L.LowbitError):
        L._heads(four[:, :2], "t")
    with pytest.raises(L.LowbitError):
        L._heads(four.transpose(-1, -2), "t")
    assert L._heads(four[:, :1], "t") == (2, 120, 8)                # a step of 120 between batches


def test_windows_beyond_64_bits():
    q = torch.zeros(4, 1, 8)
    for window in (2 ** 63, 2 ** 70):
        p = L._attention_params(q, q, q, None, None, None, True, window, None, 0.0, None)
        assert p.window == 1 << 40
    assert L._attention_params(q, q, q, None, None, None, True, -2 ** 70, None, 0.0, None).window < 0


# ----------------------------------------------------------- orthogonalize --
def _ortho(g=OK16, out=ctypes.c_void_p(0x100000), ws=OK16, bytes=1 << 50, **change):
    v = dict(batch=2, rows=30, cols=40, type=0, steps=5, a=3.0, b=-4.0, c=2.0, eps=1e-7, scale=1.0)
    v.update(change)
    return L.lib().lowbit_orthogonalize(g, L.OrthogonalizeParams(*v.values()), out, ws, bytes, None)


def test_orthogonalize_refusals():
    for bad in (dict(batch=-1), dict(batch=(1 << 20) + 1), dict(rows=0), dict(rows=65537),
                dict(cols=0), dict(cols=65537), dict(batch=1 << 20, rows=2048, cols=2048),
                dict(type=2), dict(steps=-1), dict(steps=65), dict(a=math.nan), dict(b=math.inf),
                dict(c=math.nan), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf),
                dict(scale=math.nan), dict(g=None), dict(g=OFF), dict(out=None), dict(out=OFF),
                dict(ws=None), dict(ws=OFF), dict(bytes=1000), dict(out=OK16)):
        assert _ortho(**bad) == L.EINVAL, bad
    assert _ortho(batch=0, g=None, out=None, ws=None) == L.OK
    ws = L.lib().lowbit_orthogonalize_workspace
    assert ws(None) == -1 and ws(L.OrthogonalizeParams(1, 0, 3, 0, 5, 1, 1, 1, 0, 1)) == -1
    assert ws(L.OrthogonalizeParams(2, 30, 40, 0, 5, 1, 1, 1, 0, 1)) > 2 * 30 * 40 * 10
    g = torch.zeros(3, 4)
    for call in (lambda: L.orthogonalize(g), lambda: L.orthogonalize(g[0]),
                 lambda: L.orthogonalize(g.half()), lambda: L.orthogonalize(g, out=g),
                 lambda: L.orthogonalize(g, steps=-1)):
        with pytest.raises(L.LowbitError):
            call()


def test_calls_outside_torchs_graph_are_warned_of():
    x = torch.zeros(4, 2, 8, requires_grad=True)
    f = torch.zeros(4, dtype=torch.float64)
    for call in (lambda: L.rotary(x, f), lambda: L.attention(x, x.detach(), x.detach()),
                 lambda: L.attention(x.detach(), x, x.detach()), lambda: L.orthogonalize(x)):
        with pytest.warns(UserWarning, match="gradient"), pytest.raises(L.LowbitError):
            call()


# ------------------------------------------------------------ plain forms --
@pytest.mark.parametrize("how", [dict(), dict(causal=False, window=4), dict(window=3, prefix=[2, 5]),
                                 dict(softcap=1.5, slopes=[0.1, 0.3, 0.0, 1.0])])
def test_reference_attention_gradient(how):
    """The 64-bit gradient against torch's own differentiation of the formula."""
    g = torch.Generator().manual_seed(1)
    lens, klens, h, kv, d = [7, 5], [9, 3], 4, 2, 6
    q, k, v, w = (torch.randn(n, m, d, generator=g, dtype=torch.float64, requires_grad=True)
                  for n, m in ((12, h), (12, kv), (12, kv), (12, h)))
    qb, kb = torch.tensor([0, 7, 12]), torch.tensor([0, 9, 12])
    how = {n: torch.tensor(t) if n in ("prefix", "slopes") else t for n, t in how.items()}

    outs = []
    for (q0, q1), (k0, k1), s in zip(((0, 7), (7, 12)), ((0, 9), (9, 12)), (0, 1)):
        see, far = R.visible(q1 - q0, k1 - k0, how.get("causal", True), how.get("window", 0),
                             int(how["prefix"][s]) if "prefix" in how else 0)
        for i in range(h):
            x = 0.7 * q[q0:q1, i] @ k[k0:k1, i // 2].T
            if "softcap" in how:
                x = how["softcap"] * torch.tanh(x / how["softcap"])
            if "slopes" in how:
                x = x - how["slopes"][i].double() * far
            p = torch.where(see, x, -torch.inf)
            some = see.any(1)
            o = torch.zeros(q1 - q0, d, dtype=torch.float64)
            o = torch.cat([o[:int((~some).sum())], torch.softmax(p[some], 1) @ v[k0:k1, i // 2]])
            outs.append((w[q0:q1, i] * o).sum())
    want = torch.autograd.grad(sum(outs), (q, k, v))
    t = [x.detach() for x in (q, k, v)]
    fwd, _ = R.attention(*t, qb, kb, 0.7, **how)
    assert np.isclose(float((fwd["out"] * w.detach()).sum()), float(sum(outs).detach()))
    got, _ = R.attention(*t, qb, kb, 0.7, dout=w.detach(), out=fwd["out"], lse=fwd["lse"], **how)
    for name, grad in zip(("dq", "dk", "dv"), want):
        assert torch.allclose(got[name], grad, rtol=1e-10, atol=1e-12), name


def test_reference_rotary_is_a_rotation():
    x = torch.randn(5, 2, 10, dtype=torch.float64)
    f = torch.tensor([1.0, 0.1, 0.01], dtype=torch.float64)
    for layout in ("half", "interleaved"):
        y, _ = R.rotary(x, f, torch.arange(5) * 100, layout, 1.0)
        assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1))
        z, _ = R.rotary(y, f, torch.arange(5) * 100, layout, 1.0, back=True)
        assert torch.allclose(z, x)


def test_reference_newton_schulz_acts_on_singular_values():
    g = torch.randn(6, 9, dtype=torch.float64)
    u, s, vh = torch.linalg.svd(g, full_matrices=False)
    a, b, c = 3.4445, -4.7750, 2.0315
    t = s / torch.linalg.vector_norm(s)
    for _ in range(5):
        t = a * t + b * t ** 3 + c * t ** 5
    want = u @ torch.diag(t) @ vh
    assert torch.allclose(R.newton_schulz(g, 5, (a, b, c), 0.0, 1.0), want, atol=1e-10)
    assert torch.allclose(R.newton_schulz(g.T, 5, (a, b, c), 0.0, 1.0), want.T, atol=1e-10)
