"""rotary, attention and orthogonalize where offsets pass 32 bits, on two streams at once, and of
inputs that are the same tensor."""
import pytest
import torch

pytestmark = pytest.mark.gpu
L = pytest.importorskip("weight_communication_compression_amd.lowbit")


def spread(t, row):
    """t's values with rows `row` elements apart."""
    buf = torch.empty(t.shape[0], row, dtype=t.dtype, device="cuda")
    view = buf[:, :t.shape[1] * t.shape[2]].view(t.shape[0], t.shape[1], t.shape[2])
    view.copy_(t)
    return view


def test_attention_with_rows_far_apart():
    """2200 rows 2^20 elements apart: offsets beyond 2^31 elements and 2^32 bytes."""
    g = torch.Generator().manual_seed(1)
    q, k, v, dout = (torch.randn(2200, h, 64, generator=g).bfloat16().cuda() for h in (2, 1, 1, 2))
    begin = torch.tensor([0, 100, 2200], dtype=torch.int32).cuda()
    want = L.attention(q, k, v, q_begin=begin)
    grads = L.attention_backward(dout, q, k, v, want.out, want.lse, q_begin=begin)
    far = [spread(t, 1 << 20) for t in (q, k, v)]
    got = L.attention(*far, q_begin=begin, out=spread(want.out * 0, 1 << 20))
    assert torch.equal(got.out, want.out) and torch.equal(got.lse, want.lse)
    del far[1:]
    outs = [spread(t * 0, 1 << 20) for t in (q, k, v)]
    back = L.attention_backward(dout, far[0], k, v, got.out, got.lse, q_begin=begin, dq=outs[0],
                                dk=outs[1], dv=outs[2])
    assert all(torch.equal(a, b) for a, b in zip(back, grads))


def test_attention_over_many_rows():
    """Tokens times heads times width beyond 2^31: the last document as if it were alone."""
    rows, heads = (1 << 31) // (16 * 64) + 5000, 16
    qkv = torch.empty(rows, heads + 2, 64, dtype=torch.bfloat16, device="cuda")
    tail = 300
    last = torch.randn(tail, heads + 2, 64, device="cuda").bfloat16()
    qkv[-tail:] = last
    begin = torch.tensor([rows - tail, rows], dtype=torch.int32).cuda()
    out = torch.empty(rows, heads, 64, dtype=torch.bfloat16, device="cuda")
    got = L.attention(qkv[:, :heads], qkv[:, heads:-1], qkv[:, -1:], q_begin=begin, out=out)
    want = L.attention(last[:, :heads], last[:, heads:-1], last[:, -1:])
    assert torch.equal(out[-tail:], want.out) and torch.equal(got.lse[:, -tail:], want.lse)


def test_rotary_over_many_elements():
    rows = (1 << 31) // 512 + 3
    x = torch.empty(rows, 8, 64, dtype=torch.bfloat16, device="cuda")
    last = torch.randn(5, 8, 64, device="cuda").bfloat16()
    x[-5:] = last
    freqs = L.rotary_frequencies(64)[0].cuda()
    at = torch.arange(rows, device="cuda") % 4096
    L.rotary(x, freqs, at, out=x)
    assert torch.equal(x[-5:], L.rotary(last, freqs, at[-5:].clone()))


def test_orthogonalize_many_elements():
    g = torch.zeros(2100, 1024, 1024, dtype=torch.bfloat16, device="cuda")
    g[-1] = torch.randn(1024, 1024, device="cuda")
    got = L.orthogonalize(g, steps=1, out=g.clone())
    assert torch.equal(got[-1], L.orthogonalize(g[-1].clone(), steps=1)) and (got[0] == 0).all()


def test_two_streams_at_once():
    q, k, v = (torch.randn(700, h, 128, device="cuda").bfloat16() for h in (4, 1, 1))
    m = torch.randn(300, 500, device="cuda")
    want, ortho = L.attention(q, k, v), L.orthogonalize(m)
    dout = torch.randn_like(q)
    grads = L.attention_backward(dout, q, k, v, want.out, want.lse)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    results = []
    for turn in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                a = L.attention(q, k, v)
                results.append((a, L.attention_backward(dout, q, k, v, a.out, a.lse), L.orthogonalize(m)))
    torch.cuda.synchronize()
    for a, b, o in results:
        assert torch.equal(a.out, want.out) and torch.equal(a.lse, want.lse) and torch.equal(o, ortho)
        assert all(torch.equal(x, y) for x, y in zip(b, grads))


def test_two_graphs_that_share_a_workspace():
    q, k, v = (torch.randn(300, h, 64, device="cuda") for h in (2, 1, 1))
    dout = torch.randn_like(q)
    want = L.attention(q, k, v)
    grads = L.attention_backward(dout, q, k, v, want.out, want.lse)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    graphs, kept = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            a = L.attention(q, k, v, workspace=ws)
            kept.append((a, L.attention_backward(dout, q, k, v, a.out, a.lse, workspace=ws)))
        graphs.append(graph)
    for turn in range(3):
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        ws.fill_(255)                                 # nothing in it is kept from call to call
        for a, b in kept:
            assert torch.equal(a.out, want.out)
            assert all(torch.equal(x, y) for x, y in zip(b, grads))


def test_keys_that_are_values():
    q, k = torch.randn(90, 2, 64, device="cuda"), torch.randn(90, 2, 64, device="cuda")
    assert torch.equal(L.attention(q, k, k).out, L.attention(q, k, k.clone()).out)
    got, want = L.attention(k, k, k), L.attention(k.clone(), k, k.clone())
    assert torch.equal(got.out, want.out)
