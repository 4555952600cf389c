"""rotary and its gradient against the 64-bit form."""
import pytest
import torch

import block_ref as R
from train_ref import U, half_step

pytestmark = pytest.mark.gpu
L = pytest.importorskip("weight_communication_compression_amd.lowbit")


def make(rows, heads, dim, dtype, seed=0, extra=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, heads + extra, dim, generator=g).to(dtype).cuda()
    return x[:, :heads]


def bound(x, size, want, dtype):
    # half a turn is rounded to binary32 (2^-25 of a turn's half: pi 2^-25), sine and cosine are
    # good to 2 U, two products and a sum: 8 U of what is added up
    return half_step(dtype) * want.abs() + 8 * U * size


def check(x, freqs, positions, layout="half", scale=1.0, back=False, **more):
    call = L.rotary_backward if back else L.rotary
    got = call(x, freqs.cuda(), None if positions is None else positions.cuda(), layout=layout,
               scale=scale, **more)
    at = positions
    if at is None:
        at = torch.arange(x.shape[0]) % (more.get("rows_per_sequence") or max(x.shape[0], 1))
    want, size = R.rotary(x.cpu().double(), freqs, at, layout, scale, back)
    R.close(got, want, bound(x, size, want, x.dtype), f"{x.shape} {layout}")
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rows,heads,dim,rot", [
    (1, 1, 64, 64), (3, 10, 64, 64), (7, 5, 128, 128), (130, 3, 80, 40), (5, 2, 2, 2),
    (9, 3, 96, 22), (33, 40, 128, 64), (4, 1, 257, 254), (2, 3, 30, 18)])
def test_values(rows, heads, dim, rot, layout, dtype):
    freqs, scale = L.rotary_frequencies(rot)
    at = torch.randint(0, 5000, (rows,), generator=torch.Generator().manual_seed(rows))
    x = make(rows, heads, dim, dtype, extra=2)
    check(x, freqs, at, layout, scale)
    check(x, freqs, at, layout, 1.25, back=True)


def test_far_and_negative_positions():
    freqs, scale = L.rotary_frequencies(64, scaling="parts", factor=16.0, original_length=4096)
    at = torch.tensor([0, -1, -70000, 1 << 20, (1 << 30) - 3])
    check(make(5, 3, 64, torch.float32)[:4], freqs, at[:4], "half", scale)
    # 2^30: 2^-22 of a turn
    x = make(5, 3, 64, torch.float32)
    got = L.rotary(x, freqs.cuda(), at.cuda())
    want, size = R.rotary(x.cpu().double(), freqs, at, "half", 1.0)
    R.close(got, want, 8 * U * size + 2 ** -22 * 6.2832 * size + U * want.abs(), "2^30")


def test_counted_positions():
    freqs, _ = L.rotary_frequencies(32)
    x = make(50, 2, 32, torch.bfloat16)
    check(x, freqs, None)
    check(x, freqs, None, rows_per_sequence=7)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_in_place_leaves_the_rest(layout):
    freqs, _ = L.rotary_frequencies(48)
    buf = torch.randn(37, 9, 80, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    before = buf.clone()
    at = torch.arange(37).cuda()
    want = L.rotary(before[:, 2:6], freqs.cuda(), at, layout=layout)
    got = L.rotary(buf[:, 2:6], freqs.cuda(), at, layout=layout, out=buf[:, 2:6])
    assert got.data_ptr() == buf[:, 2:6].data_ptr()
    assert torch.equal(buf[:, 2:6], want)
    assert torch.equal(buf[:, :2], before[:, :2]) and torch.equal(buf[:, 6:], before[:, 6:])


def test_turning_back_and_gradient_by_differences():
    freqs, _ = L.rotary_frequencies(64)
    x = make(11, 3, 64, torch.float32)
    y = L.rotary(x, freqs.cuda(), scale=1.5)
    # the map is linear: its transpose is exact against a difference of any size
    dy = make(11, 3, 64, torch.float32, seed=3)
    dx = L.rotary_backward(dy, freqs.cuda(), scale=1.5)
    a, b = (dy.double() * y.double()).sum(), (dx.double() * x.double()).sum()
    size = (dy.double().abs() * (y.double().abs() + 1)).sum()
    assert abs(a - b) <= 64 * U * size


def test_any_alignment_and_strides():
    freqs, _ = L.rotary_frequencies(6)
    for shift in range(4):
        flat = torch.randn(4000, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
        x = flat[shift:].as_strided((9, 4, 11), (97, 13, 1))
        check(x, freqs, torch.arange(9))
    # heads outermost
    x = torch.randn(3, 20, 16).cuda().transpose(0, 1)
    f16 = L.rotary_frequencies(16)[0]
    check(x, f16, torch.arange(20))
    out = torch.empty(3, 20, 16, device="cuda").transpose(0, 1)
    check(x, f16, torch.arange(20), out=out)


def test_no_rows_and_leading_dimensions():
    freqs, _ = L.rotary_frequencies(16)
    assert L.rotary(torch.empty(0, 2, 16, device="cuda"), freqs.cuda()).shape == (0, 2, 16)
    x = torch.randn(2, 5, 3, 16).cuda()
    got = L.rotary(x, freqs.cuda(), rows_per_sequence=5)
    want, size = R.rotary(x.cpu().double().view(10, 3, 16), freqs, torch.arange(10) % 5, "half", 1.0)
    R.close(got.view(10, 3, 16), want, U * want.abs() + 8 * U * size, "4 dimensions")


def test_other_stream_and_graph():
    freqs, _ = L.rotary_frequencies(128)
    freqs = freqs.cuda()
    x = make(100, 6, 128, torch.bfloat16)
    want = L.rotary(x, freqs)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = L.rotary(x, freqs)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.rotary(x, freqs, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
