"""orthogonalize against its 64-bit form."""
import math

import pytest
import torch

import block_ref as R
from train_ref import half_step

pytestmark = pytest.mark.gpu
L = pytest.importorskip("weight_communication_compression_amd.lowbit")
ABC = (3.4445, -4.7750, 2.0315)


def matrix(rows, cols, seed, dtype=torch.float32, rank=None, batch=()):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*batch, rows, cols, generator=g)
    if rank:
        x = 0.1 * x + torch.randn(*batch, rows, rank, generator=g) @ torch.randn(*batch, rank, cols, generator=g)
    return (x * 0.03).to(dtype)


def check(g, steps=5, scale=1.0, eps=1e-7, abc=ABC):
    got = L.orthogonalize(g.cuda(), steps=steps, scale=scale, eps=eps, coefficients=abc).cpu()
    assert got.dtype == torch.bfloat16 and got.shape == g.shape
    flat, out = g.reshape(-1, *g.shape[-2:]), got.reshape(-1, *g.shape[-2:]).double()
    for x, y in zip(flat.double(), out):
        want = R.newton_schulz(x, steps, abc, eps, scale)
        same = R.newton_schulz(x, steps, abc, eps, scale, R.to_f16)
        # the operands' roundings to binary16 leave an error of the size of the emulated one (the
        # kernel's binary32 sums may turn some of them the other way: twice that, and the sums' own
        # 2^-20); then half a step of the result
        size = torch.linalg.vector_norm(want)
        bound = 2 * torch.linalg.vector_norm(same - want) + (2 ** -20 + half_step(torch.bfloat16)) * size
        assert torch.linalg.vector_norm(y - want) <= bound, f"{x.shape} {steps}"
    return got


@pytest.mark.parametrize("rows,cols", [
    (1, 1), (1, 7), (9, 1), (2, 3), (16, 16), (31, 65), (64, 64), (65, 63), (100, 300), (128, 512),
    (130, 129), (300, 70), (257, 513), (640, 200)])
def test_sizes(rows, cols):
    check(matrix(rows, cols, rows))
    check(matrix(rows, cols, rows + 1, torch.bfloat16), scale=0.3)


@pytest.mark.parametrize("steps", [0, 1, 2, 6, 9])
def test_steps(steps):
    check(matrix(70, 90, steps), steps=steps)
    check(matrix(90, 70, steps, torch.bfloat16), steps=steps)


def test_low_rank_and_batches():
    check(matrix(200, 150, 1, rank=5))
    check(matrix(150, 260, 2, torch.bfloat16, rank=40, batch=(3,)))
    check(matrix(40, 33, 3, batch=(2, 4)))
    # matrices of a batch do not meet: each as alone
    g = matrix(70, 130, 4, batch=(5,)).cuda()
    every = L.orthogonalize(g)
    assert all(torch.equal(every[i], L.orthogonalize(g[i].contiguous())) for i in range(5))


def test_large():
    check(matrix(1100, 1500, 5, torch.bfloat16))
    check(matrix(1300, 500, 6))


@pytest.mark.parametrize("batch,rows,cols", [
    (1, 100, 5000), (1, 200, 9000), (3, 70, 3000), (1, 4100, 64), (2, 640, 640), (1, 1500, 1300),
    (1, 2100, 2000), (40, 130, 140)])
def test_every_form(batch, rows, cols):
    """Sizes that take each form of the products, some cut along k; against the form in 64 bits on
    the GPU (the same bound as above)."""
    g = matrix(rows, cols, batch + rows, batch=(batch,)).cuda()
    got = L.orthogonalize(g).double()
    for i in {0, batch - 1}:
        x = g[i].double()
        want = R.newton_schulz(x, 5, ABC, 1e-7, 1.0)
        same = R.newton_schulz(x, 5, ABC, 1e-7, 1.0, R.to_f16)
        bound = 2 * torch.linalg.vector_norm(same - want) + \
            (2 ** -20 + half_step(torch.bfloat16)) * torch.linalg.vector_norm(want)
        assert torch.linalg.vector_norm(got[i] - want) <= bound


def test_singular_values():
    s = torch.linalg.svdvals(L.orthogonalize(matrix(256, 512, 7).cuda()).float())
    assert s.max() < 1.25 and s.min() > 0.6


def test_coefficients():
    check(matrix(60, 80, 8), steps=12, abc=(1.875, -1.25, 0.375))


def test_range_of_the_input():
    g = matrix(60, 80, 9)
    want = L.orthogonalize(g.cuda())
    for factor in (2.0 ** 100, 2.0 ** -80):           # eps is of no account beside 2^-80
        got = L.orthogonalize((g * factor).cuda(), eps=0.0)
        assert (got.float() - want.float()).abs().max() <= 2 ** -7
    # zeros; a value that is not finite
    assert (L.orthogonalize(torch.zeros(20, 30, device="cuda")) == 0).all()
    bad = matrix(20, 30, 10, batch=(3,)).cuda()
    bad[1, 4, 5] = math.inf
    got = L.orthogonalize(bad)
    assert got[1].isnan().all() and got[0].isfinite().all() and got[2].isfinite().all()


def test_in_place_streams_and_graphs():
    g = matrix(130, 200, 11, torch.bfloat16).cuda()
    want = L.orthogonalize(g)
    same = g.clone()
    assert L.orthogonalize(same, out=same) is same and torch.equal(same, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = L.orthogonalize(g)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.orthogonalize(g, out=out)
    for seed in (12, 13, 14):
        g.copy_(matrix(130, 200, seed, torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, L.orthogonalize(g))


def test_nothing_to_do():
    assert L.orthogonalize(torch.empty(0, 5, 6, device="cuda")).shape == (0, 5, 6)
    assert L.orthogonalize(torch.empty(4, 0, device="cuda")).shape == (4, 0)
