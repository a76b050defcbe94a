"""The gradient of combine and dispatch on more tokens than one launch has
threads for.  Nearly all pairs are dropped (their rows would not fit), and
live ones sit on both sides of where a launch ends, at the first and at the
last token.  The values are whole numbers, so every sum is exact."""

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
K, E = 16, 16


@pytest.fixture(scope="module")
def moe():
    import combine_moe_dispatch_layout_amd as m
    m.load_library()
    assert torch.cuda.is_available()
    return m


def spots(bs, k, edges):
    """Live pairs: a few tokens around each edge, any of the k places."""
    tokens = sorted({t for at in edges for t in (at - 1, at, at + 1) if 0 <= t < bs})
    return [(t, (5 * i + 3) % k) for i, t in enumerate(tokens)]


def routes(bs, k, live, cap):
    """ids and ranks with only `live` pairs kept, pair i at row cap - 1 - i."""
    ids = torch.zeros((bs, k), dtype=torch.int32, device=DEV)
    idx = torch.full((bs * k,), -1, dtype=torch.int32, device=DEV)
    send = torch.arange(E + 1, dtype=torch.int32, device=DEV)
    for i, (t, j) in enumerate(live):
        ids[t, j] = i % E
        idx[t * k + j] = cap - 1 - i - i % E
    return ids, idx, send


@pytest.mark.parametrize("bs,hidden", [((1 << 21) + 3, 2080), ((1 << 23) + 3, 256),
                                       ((1 << 25) + 3, 64)])
def test_combine_backward_beyond_one_launch(moe, bs, hidden):
    """128, 32 and 8 threads a pair: 2^32 of them and more."""
    live = spots(bs, K, (0, 1 << 20, 1 << 21, 7 << 20, 1 << 23, 1 << 25, bs - 1))
    cap = len(live) + E
    gen = torch.Generator().manual_seed(hidden)
    ids, idx, send = routes(bs, K, live, cap)
    y = torch.randint(-3, 4, (cap, hidden), generator=gen).to(DEV, torch.bfloat16)
    g = torch.zeros((bs, hidden), dtype=torch.bfloat16, device=DEV)
    w = torch.zeros((bs, K), device=DEV)
    for t, j in live:
        g[t] = torch.randint(-3, 4, (hidden,), generator=gen).to(DEV, torch.bfloat16)
        w[t, j] = float(torch.randint(1, 9, (1,), generator=gen))
    dw = torch.full((bs, K), -1.0, device=DEV)
    dy = torch.full((cap, hidden), -5.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_combine_backward(g, y, ids, idx, send, w, E, grad_expand_x=dy,
                             grad_expert_scales=dw, check=True)
    want = torch.full((cap, hidden), -5.0, dtype=torch.bfloat16, device=DEV)
    for i, (t, j) in enumerate(live):
        row = cap - 1 - i
        want[row] = (w[t, j] * g[t].float()).bfloat16()
        assert float(dw[t, j]) == float((g[t].double() * y[row].double()).sum()), (t, j)
        dw[t, j] = 0.0
    assert torch.equal(dy, want)
    assert not dw.any()


@pytest.mark.parametrize("bs,hidden,k", [((1 << 25) + 3, 32, 1), ((1 << 24) + 3, 992, 1),
                                         ((1 << 23) + 3, 1056, 2)])
def test_dispatch_backward_and_combine_beyond_one_launch(moe, bs, hidden, k):
    """128 threads a token and 1024 channels: 2^31 and 2^32 of them and more.
    The combine with weights of two and a shared row runs on the same routes."""
    live = spots(bs, k, (0, 1 << 22, 1 << 23, 1 << 24, 1 << 25, bs - 1))
    cap = len(live) + E
    gen = torch.Generator().manual_seed(hidden)
    ids, idx, send = routes(bs, k, live, cap)
    rows = torch.randint(-3, 4, (cap, hidden), generator=gen).to(DEV, torch.bfloat16)
    add = torch.zeros((bs, hidden), dtype=torch.bfloat16, device=DEV)
    for t, j in live:
        add[t] = torch.randint(-3, 4, (hidden,), generator=gen).to(DEV, torch.bfloat16)
    out = torch.full((bs, hidden), -5.0, dtype=torch.bfloat16, device=DEV)
    w = torch.full((bs, k), 2.0, device=DEV)
    for times in (1.0, 2.0):
        out.fill_(-5.0)
        if times == 1.0:
            moe.moe_dispatch_backward(rows, ids, idx, send, E, grad_x_add=add, out=out, check=True)
        else:
            moe.moe_combine(rows, ids, idx, send, w, add, E, out=out, check=True)
        for i, (t, j) in enumerate(live):
            want = times * rows[cap - 1 - i].float() + add[t].float()
            assert torch.equal(out[t], want.bfloat16()), t
            out[t] = 0
        assert not out.any()


@pytest.mark.parametrize("bs,hidden", [(300, 64), (300, 512), (3000, 512), (3000, 1024), (70, 2080)])
def test_weights_overwritten_by_their_gradient(moe, bs, hidden):
    """grad_expert_scales may be expert_scales: a pair's weight is read before
    its gradient is written, whatever threads a pair has."""
    k, e = 4, 12
    gen = torch.Generator().manual_seed(bs + hidden)
    ids = torch.rand((bs, e), generator=gen).topk(k, 1).indices.int().to(DEV)
    lay = moe.moe_dispatch_layout(ids, e)
    cap = moe.moe_dispatch_capacity(bs, k, e)
    y = torch.randn((cap, hidden), generator=gen).to(DEV, torch.bfloat16)
    g = torch.randn((bs, hidden), generator=gen).to(DEV, torch.bfloat16)
    w = torch.rand((bs, k), generator=gen).to(DEV)
    route = (ids, lay.expand_idx, lay.ep_send_counts)
    rows = [torch.zeros((cap, hidden), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    dy, dw = moe.moe_combine_backward(g, y, *route, w, e, grad_expand_x=rows[0])
    dy2, dw2 = moe.moe_combine_backward(g, y, *route, w, e, grad_expand_x=rows[1],
                                        grad_expert_scales=w)
    assert dw2.data_ptr() == w.data_ptr()
    assert torch.equal(dw2, dw) and torch.equal(dy2, dy)
