"""Plain 64-bit forms of rotary, attention and orthogonalize, with bounds of their
rounding errors, for the tests: torch on the CPU, none of the library's code."""
import math

import numpy as np
import torch

from train_ref import U, half_step


def rotary(x, freqs, positions, layout, scale, back=False):
    """x (rows, heads, dim) float64; freqs (rot / 2), positions (rows,).  Returns the result
    and, for bounds, the size of what was added up (0 for elements that are copied)."""
    half = len(freqs)
    angle = positions.double()[:, None] * freqs * (-1 if back else 1)
    c, s = torch.cos(angle)[:, None] * scale, torch.sin(angle)[:, None] * scale
    out, size = x.clone(), torch.zeros_like(x)
    if layout == "half":
        iu, iv = slice(0, half), slice(half, 2 * half)
    else:
        iu, iv = slice(0, 2 * half, 2), slice(1, 2 * half, 2)
    u, v = x[..., iu], x[..., iv]
    out[..., iu], out[..., iv] = u * c - v * s, u * s + v * c
    size[..., iu] = size[..., iv] = (u.abs() + v.abs()) * abs(scale)
    return out, size


def lengths(begin):
    return [(int(a), int(b)) for a, b in zip(begin[:-1], begin[1:])]


def visible(lq, lk, causal, window, prefix):
    at = torch.arange(lq)[:, None] + (lk - lq)
    j = torch.arange(lk)[None]
    see = torch.ones(lq, lk, dtype=torch.bool)
    if causal:
        see &= j <= at
    if window:
        see &= (at - j).abs() < window
    return see | (j < prefix), (at - j).abs().double()


def attention(q, k, v, q_begin, k_begin, scale, causal=True, window=0, prefix=None, softcap=0.0,
              slopes=None, dtype=torch.float32, dout=None, out=None, lse=None):
    """Forward: {"out", "lse"}, each with a bound of the kernel's error.  With dout, out and lse
    (as the backward call gets them): {"dq", "dk", "dv"}.  All float64, rows by heads by dim."""
    h, kv, d = q.shape[1], k.shape[1], q.shape[2]
    weight = half_step(torch.bfloat16) if dtype == torch.bfloat16 else 0.0
    final = half_step(dtype)
    back = dout is not None
    res = {n: torch.zeros_like(t) for n, t in
           ((("dq", q), ("dk", k), ("dv", v)) if back else (("out", q),))}
    err = {n: torch.zeros_like(t) for n, t in res.items()}
    if not back:
        res["lse"] = torch.full((h, q.shape[0]), -math.inf, dtype=torch.float64)
        err["lse"] = torch.zeros(h, q.shape[0], dtype=torch.float64)
    for s, ((q0, q1), (k0, k1)) in enumerate(zip(lengths(q_begin), lengths(k_begin))):
        if q1 <= q0 or k1 <= k0:
            continue
        see, far = visible(q1 - q0, k1 - k0, causal, window, 0 if prefix is None else int(prefix[s]))
        some = see.any(1)
        for i in range(h):
            n = i // (h // kv)
            qi, ki, vi = q[q0:q1, i], k[k0:k1, n], v[k0:k1, n]
            x = scale * (qi @ ki.T)
            # a binary32 sum of d exact (binary32: rounded) products, scaled
            off = abs(scale) * (qi.abs() @ ki.abs().T) * (d + 3) * U
            y, bend, bend_off = x, torch.ones_like(x), torch.zeros_like(x)
            if softcap:
                t = torch.tanh(x / softcap)
                y, bend = softcap * t, 1 - t * t
                bend_off = 2 * off / softcap + 8 * U
                off = off + 8 * U * softcap
            if slopes is not None:
                y = y - float(slopes[i]) * far
                off = off + 3 * U * abs(float(slopes[i])) * far
            y = torch.where(see, y, torch.tensor(-math.inf, dtype=torch.float64))
            off = torch.where(see, off, torch.tensor(0.0, dtype=torch.float64))
            count = see.sum(1, keepdim=True)
            if not back:
                l = torch.logsumexp(y, 1)
                p = torch.where(some[:, None], torch.exp(y - l[:, None]), torch.tensor(0.0, dtype=torch.float64))
                p = torch.where(see, p, torch.tensor(0.0, dtype=torch.float64))
                far_from_lse = torch.where(see, (y - l[:, None]).abs(), torch.tensor(0.0, dtype=torch.float64))
                # of a weight: its score's and the maximum's error, exp's of an argument of that
                # size, the sum's
                rel = 2 * off.amax(1, keepdim=True) + (count + 24) * U \
                    + 4 * U * far_from_lse.amax(1, keepdim=True)
                o = p @ vi
                res["out"][q0:q1, i] = o
                err["out"][q0:q1, i] = (p @ vi.abs()) * (rel + weight + count * U) + final * o.abs()
                res["lse"][i, q0:q1] = l
                err["lse"][i, q0:q1] = torch.where(some, rel[:, 0] + 6 * U * l.abs() + 6 * U, torch.tensor(0.0, dtype=torch.float64))
                continue
            l = lse[i, q0:q1][:, None]
            p = torch.where(see, torch.exp(y - torch.where(l == -math.inf, 0.0, l)),
                            torch.tensor(0.0, dtype=torch.float64))
            rel = off + (24 + 4 * (torch.where(see, y.abs(), 0.0) + torch.where(l == -math.inf, 0.0, l.abs()))) * U
            do = dout[q0:q1, i]
            dp, big = do @ vi.T, do.abs() @ vi.abs().T
            delta = (do * out[q0:q1, i]).sum(1, keepdim=True)
            dbig = (do * out[q0:q1, i]).abs().sum(1, keepdim=True)
            g = p * (dp - delta) * bend
            goff = p * (dp - delta).abs() * (bend * (rel + 4 * U) + bend_off) \
                + p * bend * ((d + 3) * U * (big + dbig))
            gall = g.abs() * weight + goff * (1 + weight)
            res["dq"][q0:q1, i] = scale * (g @ ki)
            err["dq"][q0:q1, i] = abs(scale) * (gall @ ki.abs() + (count + 2) * U * (g.abs() @ ki.abs()))
            rows = see.sum(0)[:, None] + 2
            res["dk"][k0:k1, n] += scale * (g.T @ qi)
            err["dk"][k0:k1, n] += abs(scale) * (gall.T @ qi.abs() + h // kv * rows * U * (g.abs().T @ qi.abs()))
            res["dv"][k0:k1, n] += p.T @ do
            err["dv"][k0:k1, n] += (p * (rel + weight)).T @ do.abs() + h // kv * rows * U * (p.T @ do.abs())
    if back:
        for n in res:
            err[n] += final * res[n].abs()
    return res, err


def newton_schulz(g, steps, abc, eps, scale, operand=lambda t, unit: t):
    """Of one matrix (float64).  operand: how the products' operands are rounded."""
    a, b, c = abc
    x = g.T if g.shape[0] > g.shape[1] else g
    x = x / (torch.linalg.vector_norm(x) + eps)
    for _ in range(steps):
        r = operand(x, 64.0)
        gram = operand(r @ r.T, 1024.0)
        x = a * x + operand(b * gram + c * (gram @ gram), 64.0) @ r
    return scale * (x.T if g.shape[0] > g.shape[1] else x)


def to_f16(t, unit):
    return (t * unit).to(torch.float16).double() / unit


def close(got, want, bound, what):
    got, want, bound = (np.asarray(t.detach().cpu().double()) for t in (got, want, bound))
    assert got.shape == want.shape, what
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN elsewhere"
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), what
    over = np.abs(got[fine] - want[fine]) / np.maximum(bound[fine], 1e-30)
    assert not over.size or over.max() <= 1.0, \
        f"{what}: {np.sum(over > 1)} of {over.size} values off, worst {over.max():.3g} times the bound"
