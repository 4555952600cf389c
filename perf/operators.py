"""The training-step operators' workloads: what is timed, on which inputs, and
what the results have to be.

Three operators, those between which a data-parallel rank's gradients come
into being before the codec compresses them:

  dropout       y = residual + D(x), and its gradient, with a mask that is
                drawn from the library's counter hash and never stored
  block_join    what stands between two blocks of a residual network:
                x_out = a x + gate * D(norm(f)),  z = norm(x_out),
                and its gradient
  linear_xent   softmax cross entropy of x w^T over a large vocabulary, the
                logits never kept, and its gradient

``run`` computes them in elementary binary32 tensor operations, or, where
``own`` is true, by the library's calls.  ``exact`` computes them in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
IGNORED = -100
M32 = 0xFFFFFFFF


# ------------------------------------------------------------------ cases --
def listed():
    """The listed cases: real sizes from the smallest call to the largest."""
    return [
        # a single ragged activation of a few tokens: latency only
        {"name": "dropout_small", "op": "dropout", "back": False, "n": 7 * 1021, "dtype": "bf16",
         "residual": False, "p": 0.1},
        # residual add after a dropped block output, the repository's bucket size
        {"name": "dropout_add_64Mi", "op": "dropout", "back": False, "n": 1 << 26,
         "dtype": "bf16", "residual": True, "p": 0.1},
        # gradient of a binary32 activation of odd length
        {"name": "dropout_back_f32", "op": "dropout", "back": True, "n": (1 << 24) + 77,
         "dtype": "f32", "residual": False, "p": 0.25},
        # four tokens, hidden 4096: latency
        {"name": "join_small", "op": "join", "back": False, "rows": 4, "cols": 4096,
         "dtype": "bf16", "stream": "bf16", "params": "bf16", "norm": "rms", "group": 4,
         "bias": False, "p": 0.0, "scale": 1.0},
        # a micro-batch of 16 Ki tokens at the repository's hidden size, gate per channel
        {"name": "join_16Ki", "op": "join", "back": False, "rows": 16384, "cols": 4096,
         "dtype": "bf16", "stream": "bf16", "params": "bf16", "norm": "rms", "group": 16384,
         "bias": False, "p": 0.1, "scale": 1.0},
        # its gradient, gate per sequence of 2 Ki tokens
        {"name": "join_back_16Ki", "op": "join", "back": True, "rows": 16384, "cols": 4096,
         "dtype": "bf16", "stream": "bf16", "params": "bf16", "norm": "rms", "group": 2048,
         "bias": False, "p": 0.1, "scale": 1.0},
        # layer norms with biases over an odd width, binary32 residual stream under bf16 blocks
        {"name": "join_back_odd", "op": "join", "back": True, "rows": 1531, "cols": 1155,
         "dtype": "bf16", "stream": "f32", "params": "f32", "norm": "layer", "group": 7,
         "bias": True, "p": 0.2, "scale": 0.7},
        # a few tokens against a whole vocabulary: bound by reading the weights once
        {"name": "xent_small", "op": "xent", "back": False, "n": 13, "vocab": 50257, "hidden": 1024,
         "dtype": "bf16", "ignored": 0.0, "lse_grad": False},
        # the loss of a training micro-batch, hidden 4096
        {"name": "xent_8Ki", "op": "xent", "back": False, "n": 8192, "vocab": 50257,
         "hidden": 4096, "dtype": "bf16", "ignored": 0.0, "lse_grad": False},
        # its gradient where a quarter of the tokens are left out (prompts, padding)
        {"name": "xent_back_8Ki", "op": "xent", "back": True, "n": 8192, "vocab": 50257,
         "hidden": 4096, "dtype": "bf16", "ignored": 0.25, "lse_grad": False},
        # gradient over a larger vocabulary, ragged token count, z-loss
        {"name": "xent_back_128Ki", "op": "xent", "back": True, "n": 2011, "vocab": 131072,
         "hidden": 2048, "dtype": "bf16", "ignored": 0.1, "lse_grad": True},
        # binary32 master copies, odd everything
        {"name": "xent_back_f32", "op": "xent", "back": True, "n": 1023, "vocab": 10007,
         "hidden": 515, "dtype": "f32", "ignored": 0.1, "lse_grad": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["dropout", "join", "join", "xent", "xent"])
    back = rng.random() < 0.5
    p = rng.choice([0.0, 0.1, 0.2, rng.uniform(0.0, 0.9)])
    if op == "dropout":
        dtype = rng.choice(["bf16", "f32"])
        # (from 64 elements on: of fewer, a large p leaves none, whatever the inputs)
        return {"op": op, "back": back, "n": _log_int(rng, 64, 1 << (26 if dtype == "bf16" else 25)),
                "dtype": dtype, "residual": not back and rng.random() < 0.5, "p": p}
    if op == "join":
        cols = _log_int(rng, 33, 8192)
        if rng.random() < 0.7:
            cols = -(-cols // 8) * 8
        rows = _log_int(rng, 1, min(16384, (1 << 25) // cols))
        dtype, stream = rng.choice([("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
        group = rng.choice([0, 1, rows, max(1, rows // 7), rng.randint(1, rows)])
        return {"op": op, "back": back, "rows": rows, "cols": cols, "dtype": dtype,
                "stream": stream, "params": rng.choice([dtype, "f32"]),
                "norm": rng.choice(["rms", "layer"]), "group": group,
                "bias": rng.random() < 0.5, "p": p, "scale": rng.choice([1.0, 0.5])}
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    n, hidden = _log_int(rng, 1, 8192), _log_int(rng, 64, 4096)
    if rng.random() < 0.8:
        hidden = -(-hidden // 8) * 8
    most = (1 << 39) if dtype == "bf16" else (1 << 33)
    vocab = min(_log_int(rng, 1000, 131072), most // (n * hidden))
    return {"op": op, "back": back, "n": n, "vocab": max(vocab, 100), "hidden": hidden,
            "dtype": dtype, "ignored": rng.choice([0.0, 0.0, 0.1, rng.uniform(0.0, 0.8)]),
            "lse_grad": back and rng.random() < 0.3}


def _type(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _size(name):
    return {"bf16": 2, "f32": 4}[name]


def _left_out(case):
    return min(case["n"] - 1, int(case["ignored"] * case["n"]))


def work(case):
    """Each input read once, each output written once; the products and the
    elementwise arithmetic of the formulas."""
    if case["op"] == "dropout":
        streams = 3 if case["residual"] else 2
        return {"bytes": streams * case["n"] * _size(case["dtype"]),
                "flops": case["n"] * (streams - 1)}
    if case["op"] == "join":
        t, h = case["rows"], case["cols"]
        params = (3 if case["bias"] else 1) + (1 if case["bias"] else 0)
        gates = -(-t // case["group"]) if case["group"] else 0
        small = h * (params + gates) * _size(case["params"]) + 16 * t
        a, s = _size(case["dtype"]), _size(case["stream"])
        if case["back"]:  # read dx_out, dz, f, x_out; write df, dx
            return {"bytes": t * h * (3 * a + 3 * s) + small + 4 * h * (params + gates),
                    "flops": 24 * t * h}
        return {"bytes": t * h * (2 * a + 2 * s) + small, "flops": 12 * t * h}
    n, v, h, e = case["n"], case["vocab"], case["hidden"], _size(case["dtype"])
    valid = n - _left_out(case)
    if case["back"]:
        return {"bytes": 2 * e * (n + v) * h + 24 * n, "flops": 6 * valid * v * h}
    return {"bytes": e * (n + v) * h + 16 * n, "flops": 2 * valid * v * h}


# ----------------------------------------------------------------- inputs --
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.float32, std=1.0, mean=0.0):
        t = torch.randn(shape, generator=g, device=DEV)
        return t.mul_(std).add_(mean).to(dtype)

    s = dict(case)
    s["seed"] = 1000003 * seed + 17
    if case["op"] == "dropout":
        t = _type(case["dtype"])
        s["x"] = normal(case["n"], dtype=t)
        s["r"] = normal(case["n"], dtype=t) if case["residual"] else None
        return s
    if case["op"] == "join":
        t, h, dt, st, pt = (case["rows"], case["cols"], _type(case["dtype"]),
                            _type(case["stream"]), _type(case["params"]))
        # block outputs and residual streams: a few channels far larger than the rest
        loud = torch.where(torch.rand(h, generator=g, device=DEV) < 0.01, 20.0, 1.0)
        s["f"] = (normal(t, h, std=0.5) * loud).to(dt)
        s["x"] = (normal(t, h) * loud).to(st)
        s["post_w"] = normal(h, dtype=pt, std=0.1, mean=1.0)
        s["pre_w"] = normal(h, dtype=pt, std=0.1, mean=1.0) if case["bias"] else None
        s["post_b"] = normal(h, dtype=pt, std=0.1) if case["bias"] else None
        s["pre_b"] = normal(h, dtype=pt, std=0.1) if case["bias"] else None
        gates = -(-t // case["group"]) if case["group"] else 0
        s["gate"] = normal(gates, h, dtype=pt, std=0.3, mean=0.5) if gates else None
        if case["back"]:
            x_out, _, s["stats"] = _join(s, s["f"], s["x"])
            s["x_out"] = x_out
            s["dx_out"] = normal(t, h, dtype=st, std=1e-2)
            s["dz"] = normal(t, h, dtype=dt, std=1e-2)
        return s
    n, v, h, dt = case["n"], case["vocab"], case["hidden"], _type(case["dtype"])
    s["x"] = normal(n, h, dtype=dt)
    s["w"] = normal(v, h, dtype=dt, std=1.5 / math.sqrt(h))
    # tokens as they come in text: a few frequent, most rare
    u = torch.rand(n, generator=g, device=DEV, dtype=torch.float64)
    s["t"] = (torch.exp(u * math.log(v)) - 1).to(torch.int64).clamp_(0, v - 1)
    k = _left_out(case)
    if k:
        s["t"][torch.randperm(n, generator=g, device=DEV)[:k]] = IGNORED
    if case["back"]:
        s["lse"] = _xent(s["x"], s["w"], s["t"])[1]
        s["dloss"] = torch.full((n,), 1.0 / (n - k), device=DEV)
        s["dlse"] = None
        if case["lse_grad"]:  # the gradient of 1e-2 * mean(lse^2), and weights of their own for the rows
            s["dloss"] = s["dloss"] * torch.rand(n, generator=g, device=DEV)
            s["dlse"] = 2e-2 * s["lse"] / (n - k)
    return s


# ------------------------------------------------------- plain, in 32 bits --
def _fmix32(h):
    h = h ^ (h >> 16)
    h = (h * 0x85EBCA6B) & M32
    h = h ^ (h >> 13)
    h = (h * 0xC2B2AE35) & M32
    return h ^ (h >> 16)


def _key(seed):
    seed &= (1 << 64) - 1
    return _fmix32((seed & M32) ^ _fmix32((seed >> 32) ^ 0x9E3779B9))


def _keep(n, p, seed):
    """Which of n elements stay: two 16-bit draws from the hash of each pair's index."""
    pair = torch.arange((n + 1) // 2, device=DEV, dtype=torch.int64)
    word = _fmix32((pair & M32) ^ _fmix32((pair >> 32) ^ _key(seed)))
    drawn = torch.stack([word & 0xFFFF, word >> 16], 1).reshape(-1)[:n]
    return drawn >= round(p * 65536)


def _factor(p):
    left = 65536 - round(p * 65536)
    return 65536.0 / left if left else 0.0


def _dropped(x, p, seed):
    """D(x) of binary32 x; rows of a matrix begin at even draws."""
    if p == 0.0:
        return x
    if x.dim() == 2:
        rows, cols = x.shape
        wide = cols + cols % 2
        keep = _keep(rows * wide, p, seed).view(rows, wide)[:, :cols]
    else:
        keep = _keep(x.numel(), p, seed)
    return torch.where(keep, x * _factor(p), torch.zeros_like(x))


def _by_row(gate, rows, group):
    if gate is None:
        return torch.ones((), device=DEV)
    return gate.float()[torch.arange(rows, device=DEV) // group]


def _stats(x, norm, eps):
    mean = x.mean(1) if norm == "layer" else torch.zeros(x.shape[0], device=DEV)
    var = (x - mean[:, None]).square().mean(1)
    return mean, 1.0 / torch.sqrt(var + eps)


EPS = 1e-6


def _affine(xhat, w, b):
    y = xhat if w is None else xhat * w.float()
    return y if b is None else y + b.float()


def _join(s, f, x):
    f, x = f.float(), x.float()
    mean1, rstd1 = _stats(f, s["norm"], EPS)
    u = _affine((f - mean1[:, None]) * rstd1[:, None], s["post_w"], s["post_b"])
    y = s["scale"] * x + _by_row(s["gate"], s["rows"], s["group"]) * _dropped(u, s["p"], s["seed"])
    mean2, rstd2 = _stats(y, s["norm"], EPS)
    z = _affine((y - mean2[:, None]) * rstd2[:, None], s["pre_w"], s["pre_b"])
    return (y.to(_type(s["stream"])), z.to(_type(s["dtype"])),
            torch.stack([mean1, rstd1, mean2, rstd2], 1))


def _norm_back(dxhat, xhat, rstd, norm):
    m = (dxhat * xhat).mean(1, keepdim=True)
    d = dxhat - xhat * m
    if norm == "layer":
        d = d - dxhat.mean(1, keepdim=True)
    return d * rstd[:, None]


def _grouped(x, group):
    """Sums of consecutive groups of rows (the last one may be short)."""
    rows, cols = x.shape
    groups = -(-rows // group)
    wide = torch.zeros(groups * group, cols, device=DEV)
    wide[:rows] = x
    return wide.view(groups, group, cols).sum(1)


def _join_back(s):
    f, y, dz = s["f"].float(), s["x_out"].float(), s["dz"].float()
    mean1, rstd1, mean2, rstd2 = s["stats"].unbind(1)
    yhat = (y - mean2[:, None]) * rstd2[:, None]
    dyhat = dz if s["pre_w"] is None else dz * s["pre_w"].float()
    dy = s["dx_out"].float() + _norm_back(dyhat, yhat, rstd2, s["norm"])
    fhat = (f - mean1[:, None]) * rstd1[:, None]
    u = _affine(fhat, s["post_w"], s["post_b"])
    du = _dropped(dy * _by_row(s["gate"], s["rows"], s["group"]), s["p"], s["seed"])
    df = _norm_back(du if s["post_w"] is None else du * s["post_w"].float(), fhat, rstd1, s["norm"])
    out = {"df": df.to(_type(s["dtype"])), "dx": (s["scale"] * dy).to(_type(s["stream"]))}
    out["dpost_weight"] = (du * fhat).sum(0)
    if s["post_b"] is not None:
        out["dpost_bias"] = du.sum(0)
    if s["gate"] is not None:
        out["dgate"] = _grouped(dy * _dropped(u, s["p"], s["seed"]), s["group"])
    if s["pre_w"] is not None:
        out["dpre_weight"] = (dz * yhat).sum(0)
    if s["pre_b"] is not None:
        out["dpre_bias"] = dz.sum(0)
    return out


def _xent(x, w, t):
    logits = x.float() @ w.float().t()
    top = logits.max(1).values
    lse = top + torch.log(torch.exp(logits - top[:, None]).sum(1))
    counts = t != IGNORED
    hit = logits.gather(1, torch.where(counts, t, 0)[:, None])[:, 0]
    zero = torch.zeros_like(lse)
    return torch.where(counts, lse - hit, zero), torch.where(counts, lse, zero)


def _xent_back(s):
    x, w, t, dloss = s["x"].float(), s["w"].float(), s["t"], s["dloss"]
    counts = t != IGNORED
    both = dloss if s["dlse"] is None else dloss + s["dlse"]
    d = torch.exp(x @ w.t() - s["lse"][:, None]) * both[:, None]
    d.scatter_add_(1, torch.where(counts, t, 0)[:, None], -dloss[:, None])
    d = torch.where(counts[:, None], d, torch.zeros((), device=DEV))
    dt = _type(s["dtype"])
    return (d @ w).to(dt), (d.t() @ x).to(dt)


# ------------------------------------------------------------------- run ---
def _run_own(s):
    from weight_communication_compression_amd import lowbit as L
    if s["op"] == "dropout":
        if s["back"]:
            return L.dropout_backward(s["x"], s["p"], s["seed"])
        return L.dropout(s["x"], s["p"], s["seed"], residual=s["r"])
    if s["op"] == "join":
        how = dict(post_weight=s["post_w"], post_bias=s["post_b"], gate=s["gate"],
                   rows_per_gate=s["group"], pre_weight=s["pre_w"], pre_bias=s["pre_b"],
                   norm=s["norm"], residual_scale=s["scale"], eps=EPS, p=s["p"], seed=s["seed"])
        if not s["back"]:
            return tuple(L.block_join(s["f"], s["x"], **how))
        d = L.block_join_backward(s["dx_out"], s["dz"], s["f"], s["x_out"], s["stats"], **how)
        return {k: v for k, v in d._asdict().items() if v is not None}
    if not s["back"]:
        return tuple(L.linear_xent(s["x"], s["w"], s["t"], ignore_index=IGNORED))
    return tuple(L.linear_xent_backward(s["x"], s["w"], s["t"], s["lse"], s["dloss"],
                                        dlse=s["dlse"], ignore_index=IGNORED))


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "dropout":
        y = _dropped(s["x"].float(), s["p"], s["seed"])
        return (y if s["r"] is None else s["r"].float() + y).to(_type(s["dtype"]))
    if s["op"] == "join":
        return _join_back(s) if s["back"] else _join(s, s["f"], s["x"])
    return _xent_back(s) if s["back"] else _xent(s["x"], s["w"], s["t"])


# ------------------------------------------------------- exact, in 64 bits --
def _draws(count, seed):
    """uint16 draws 0 .. count-1, from numpy's wrapping 32-bit arithmetic."""
    def mix(a):
        a = a ^ (a >> np.uint32(16))
        a = a * np.uint32(0x85EBCA6B)
        a = a ^ (a >> np.uint32(13))
        a = a * np.uint32(0xC2B2AE35)
        return a ^ (a >> np.uint32(16))

    one = lambda v: np.array([v & M32], dtype=np.uint32)  # noqa: E731
    key = mix(one(seed) ^ mix(one(seed >> 32) ^ one(0x9E3779B9)))
    pairs = np.arange(-(-count // 2), dtype=np.uint32)   # below 2^32 for every case
    return mix(pairs ^ mix(key)).view("<u2")[:count]


def _mask64(shape, p, seed):
    """The factor of every element: 0, or what a kept one is multiplied by."""
    cut = round(p * 65536)
    wide = list(shape)
    wide[-1] += wide[-1] % 2
    left = _draws(math.prod(wide), seed).astype(np.int32).reshape(wide)[..., :shape[-1]] >= cut
    m = torch.from_numpy(left).to(DEV).double()
    return m * (65536.0 / (65536 - cut)) if cut < 65536 else m


def _wide_gate(s):
    if s["gate"] is None:
        return 1.0
    return s["gate"].double().repeat_interleave(s["group"], 0)[:s["rows"]]


def _or(v, other):
    return other if v is None else v.double()


def _exact_join(s):
    """Forward: the definition, through sums written as products with ones."""
    n = s["cols"]
    ones = torch.ones(n, 1, device=DEV, dtype=torch.float64)
    layer = s["norm"] == "layer"

    def normed(v, w, b):
        mean = (v @ ones) / n if layer else torch.zeros(len(v), 1, device=DEV, dtype=torch.float64)
        c = v - mean
        rstd = ((c * c) @ ones / n + EPS).rsqrt()
        return c * rstd * _or(w, 1.0) + _or(b, 0.0), mean[:, 0], rstd[:, 0]

    u, m1, r1 = normed(s["f"].double(), s["post_w"], s["post_b"])
    y = s["x"].double() * s["scale"] + u * _mask64(u.shape, s["p"], s["seed"]) * _wide_gate(s)
    z, m2, r2 = normed(y, s["pre_w"], s["pre_b"])
    return y, z, torch.stack([m1, r1, m2, r2], 1)


def _exact_join_back(s):
    n = s["cols"]
    layer = s["norm"] == "layer"
    st = s["stats"].double()

    def back(d, v, mean, rstd):
        """Gradient of a norm by the projection that it is: off the row's own direction and, centred, off the ones."""
        h = (v - mean[:, None]) * rstd[:, None]
        along = torch.linalg.vecdot(d, h)[:, None] / n
        g = d - h * along
        if layer:
            g = g - d.sum(1, keepdim=True) / n
        return g * rstd[:, None], h

    dz = s["dz"].double()
    through, yh = back(dz * _or(s["pre_w"], 1.0), s["x_out"].double(), st[:, 2], st[:, 3])
    dy = through + s["dx_out"].double()
    m = _mask64((s["rows"], n), s["p"], s["seed"])
    du = dy * _wide_gate(s) * m
    df, fh = back(du * _or(s["post_w"], 1.0), s["f"].double(), st[:, 0], st[:, 1])
    out = {"df": df, "dx": dy * s["scale"], "dpost_weight": torch.linalg.vecdot(du, fh, dim=0)}
    if s["post_b"] is not None:
        out["dpost_bias"] = du.sum(0)
    if s["gate"] is not None:
        part = dy * m * (fh * _or(s["post_w"], 1.0) + _or(s["post_b"], 0.0))
        rows = torch.arange(s["rows"], device=DEV) // s["group"]
        sums = torch.zeros(len(s["gate"]), n, device=DEV, dtype=torch.float64)
        out["dgate"] = sums.index_add_(0, rows, part)
    if s["pre_w"] is not None:
        out["dpre_weight"] = torch.linalg.vecdot(dz, yh, dim=0)
    if s["pre_b"] is not None:
        out["dpre_bias"] = dz.sum(0)
    return out


def _exact_xent(s):
    """Over valid rows alone, the vocabulary in pieces."""
    rows = torch.nonzero(s["t"] != IGNORED)[:, 0]
    x, t, step = s["x"][rows].double(), s["t"][rows], 16384
    starts = range(0, s["vocab"], step)
    if not s["back"]:
        parts = [torch.logsumexp(x @ s["w"][a:a + step].double().t(), 1) for a in starts]
        lse = torch.logsumexp(torch.stack(parts, 1), 1)
        hit = (x * s["w"][t].double()).sum(1)
        out = torch.zeros(2, s["n"], device=DEV, dtype=torch.float64)
        out[0, rows], out[1, rows] = lse - hit, lse
        return out[0], out[1]
    lse, dloss = s["lse"][rows].double(), s["dloss"][rows].double()
    both = dloss if s["dlse"] is None else dloss + s["dlse"][rows].double()
    dx = -dloss[:, None] * s["w"][t].double()
    dw = []
    for a in starts:
        w = s["w"][a:a + step].double()
        q = (x @ w.t() - lse[:, None]).exp() * both[:, None]
        dx += q @ w
        dw.append(q.t() @ x)
    dw = torch.cat(dw).index_add_(0, t, -dloss[:, None] * x)
    full = torch.zeros(s["n"], s["hidden"], device=DEV, dtype=torch.float64)
    full[rows] = dx
    return full, dw


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "dropout":
        y = s["x"].double() * _mask64(s["x"].shape, s["p"], s["seed"])
        return y if s["r"] is None else y + s["r"].double()
    if s["op"] == "join":
        return _exact_join_back(s) if s["back"] else _exact_join(s)
    return _exact_xent(s)
