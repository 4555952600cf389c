"""Plain 64-bit forms of the training-step operators, for the tests: numpy on
the CPU, none of the library's code."""
import numpy as np
import torch

U = 2.0 ** -24                       # half a step of binary32, relative


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def f64(t) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()


def fmix(h: int) -> int:
    h ^= h >> 16
    h = h * 0x85EBCA6B & 0xFFFFFFFF
    h ^= h >> 13
    h = h * 0xC2B2AE35 & 0xFFFFFFFF
    return h ^ h >> 16


def seed_key(seed: int) -> int:
    return fmix((seed & 0xFFFFFFFF) ^ fmix((seed >> 32 & 0xFFFFFFFF) ^ 0x9E3779B9))


def draws(first: int, count: int, seed: int) -> np.ndarray:
    """The 16-bit draws of mask indices first .. first + count - 1 (first even)."""
    key = seed_key(seed % 2 ** 64)
    pair = first // 2 + np.arange(-(-count // 2), dtype=np.uint64)
    hi = np.array([fmix(int(h) ^ key) for h in np.unique(pair >> np.uint64(32))], np.uint32)
    h = (pair & np.uint64(0xFFFFFFFF)).astype(np.uint32) ^ \
        hi[np.unique(pair >> np.uint64(32), return_inverse=True)[1]]
    h ^= h >> np.uint32(16)
    h *= np.uint32(0x85EBCA6B)
    h ^= h >> np.uint32(13)
    h *= np.uint32(0xC2B2AE35)
    h ^= h >> np.uint32(16)
    return np.stack([h & np.uint32(0xFFFF), h >> np.uint32(16)], 1).reshape(-1)[:count]


def cut_and_factor(p: float):
    cut = round(p * 65536)
    return cut, (65536.0 / (65536 - cut) if cut < 65536 else 0.0)


def keep_rows(rows: int, cols: int, p: float, seed: int) -> np.ndarray:
    wide = cols + cols % 2
    return (draws(0, rows * wide, seed) >= cut_and_factor(p)[0]).reshape(rows, wide)[:, :cols]


def norm_stats(v, norm, eps):
    mean = v.mean(1) if norm == "layer" else np.zeros(len(v))
    return mean, 1 / np.sqrt(((v - mean[:, None]) ** 2).mean(1) + eps)


def join(f, x, post_w, post_b, gate, group, pre_w, pre_b, norm, a, eps, p, seed):
    """All arrays float64 (or None).  Returns x_out, z, stats and, for bounds,
    the size of what was added up for x_out."""
    m1, r1 = norm_stats(f, norm, eps)
    fh = (f - m1[:, None]) * r1[:, None]
    w, b = (1.0 if post_w is None else post_w), (0.0 if post_b is None else post_b)
    u = fh * w + b
    keep = keep_rows(*f.shape, p, seed)
    factor = cut_and_factor(p)[1]
    g = 1.0 if gate is None else gate[np.arange(len(f)) // group]
    y = a * x + g * np.where(keep, u * factor, 0.0)
    size = np.abs(a * x) + np.abs(g) * keep * factor * (
        (np.abs(f) + np.abs(f).mean(1, keepdims=True)) * r1[:, None] * np.abs(w) + np.abs(b))
    m2, r2 = norm_stats(y, norm, eps)
    z = (y - m2[:, None]) * r2[:, None] * (1.0 if pre_w is None else pre_w) \
        + (0.0 if pre_b is None else pre_b)
    return y, z, np.stack([m1, r1, m2, r2], 1), size


def norm_back(d, xh, rstd, norm):
    g = d - xh * (d * xh).mean(1, keepdims=True)
    if norm == "layer":
        g = g - d.mean(1, keepdims=True)
    return g * rstd[:, None]


def join_back(dxo, dz, f, y, stats, post_w, post_b, gate, group, pre_w, norm, a, p, seed):
    """Gradients, and per gradient the size of what was added up for it."""
    m1, r1, m2, r2 = stats.T
    yh = (y - m2[:, None]) * r2[:, None]
    q = dz * (1.0 if pre_w is None else pre_w)
    dy = dxo + norm_back(q, yh, r2, norm)
    w, b = (1.0 if post_w is None else post_w), (0.0 if post_b is None else post_b)
    fh = (f - m1[:, None]) * r1[:, None]
    u = fh * w + b
    m = keep_rows(*f.shape, p, seed) * cut_and_factor(p)[1]
    groups = np.arange(len(f)) // group if gate is not None else None
    g = 1.0 if gate is None else gate[groups]
    du = m * g * dy
    df = norm_back(du * w, fh, r1, norm)

    def sums(v):
        return v.sum(0), np.abs(v).sum(0)

    # sizes: the rows' own roundings, |dy| taken as what it is the sum of
    yha = (np.abs(y) + np.abs(m2)[:, None]) * r2[:, None]
    fha = (np.abs(f) + np.abs(m1)[:, None]) * r1[:, None]
    qa = np.abs(q)
    dya = np.abs(dxo) + r2[:, None] * (qa + yha * (qa * yha).mean(1, keepdims=True)
                                       + qa.mean(1, keepdims=True))
    dua = m * np.abs(g) * dya
    sa = dua * np.abs(w)
    dfa = r1[:, None] * (sa + fha * (sa * fha).mean(1, keepdims=True) + sa.mean(1, keepdims=True))
    ua = fha * np.abs(w) + np.abs(b)
    out = {"df": (df, dfa), "dx": (a * dy, abs(a) * dya),
           "dpost_weight": ((du * fh).sum(0), (dua * fha).sum(0)),
           "dpost_bias": (du.sum(0), dua.sum(0)),
           "dpre_weight": ((dz * yh).sum(0), (np.abs(dz) * yha).sum(0)),
           "dpre_bias": sums(dz)}
    if gate is not None:
        part, size = dy * m * u, dya * m * ua
        out["dgate"] = tuple(np.stack([v[groups == k].sum(0) for k in range(groups[-1] + 1)])
                             for v in (part, size))
    return out


def within(got, want, bound, what):
    """|got - want| <= bound everywhere (and NaN or infinite where want is)."""
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), what
    bound = np.broadcast_to(bound, want.shape)
    over = np.abs(got - want)[fine] / np.maximum(bound[fine], 1e-300)
    assert not over.size or over.max() <= 1.0, \
        f"{what}: {np.sum(over > 1)} of {over.size} values off, worst {over.max():.3g} times the bound"
