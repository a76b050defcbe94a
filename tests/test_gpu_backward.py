"""The gradient of combine and dispatch on the GPU.

Bars, from the arithmetic alone: grad_expand_x is one fp32 product rounded
to bf16, so it equals that rounding bit for bit; grad_expert_scales is an fp32
sum of H products, off by at most (H + 1) * 2^-24 of the terms' summed
magnitude; grad_x is an fp32 sum in fixed order rounded once, bit for bit.
Both gradients are also compared with difference quotients of the 64-bit
forward.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
SENTINEL = -12345.0   # exact in bf16


@pytest.fixture(scope="module")
def moe():
    import combine_moe_dispatch_layout_amd as m
    m.load_library()
    assert torch.cuda.is_available()
    return m


class Case:
    """Inputs on the CPU, with the layout they have, and copies on the GPU."""

    def __init__(self, moe, bs, hidden, e, k, *, dropped=0.0, repeat=False, align=128, seed=0,
                 pad=0):
        gen = torch.Generator().manual_seed(seed)
        self.bs, self.hidden, self.e, self.k = bs, hidden, e, k
        ids = torch.rand((bs, e), generator=gen).topk(k, 1).indices.int()
        if repeat:
            ids[:, -1] = ids[:, 0]
        drop = torch.rand((bs, k), generator=gen) < dropped
        ids[drop] = torch.where(torch.rand((bs, k), generator=gen) < 0.5, -1, e)[drop].int()
        self.ids = ids
        lay = moe.moe_dispatch_layout(ids.to(DEV), e, align)
        self.idx, self.send = lay.expand_idx.cpu(), lay.ep_send_counts.cpu()
        self.cap = max(int(self.send[-1]), 1)
        self.real = ((ids >= 0) & (ids < e)).reshape(-1)
        self.slot = (self.send[ids.clamp(0, e - 1).long()].reshape(-1) + self.idx).long()
        self.w = torch.softmax(torch.randn((bs, k), generator=gen), 1)
        self.g = torch.randn((bs, hidden), generator=gen).bfloat16()
        self.rows = torch.randn((self.cap, hidden), generator=gen).bfloat16()
        self.add = torch.randn((bs, hidden), generator=gen).bfloat16()
        self.pad = pad
        self.route = (ids.to(DEV), lay.expand_idx, lay.ep_send_counts)

    def on(self, t):
        if not self.pad:
            return t.to(DEV)
        buf = torch.full((t.shape[0], t.shape[1] + self.pad), 77.0, dtype=t.dtype, device=DEV)
        buf[:, :t.shape[1]] = t.to(DEV)
        return buf[:, :t.shape[1]]


def check_combine_backward(moe, c):
    out = c.on(torch.full((c.cap, c.hidden), SENTINEL, dtype=torch.bfloat16))
    dw = torch.full((c.bs, c.k), SENTINEL, device=DEV)
    dy, dw = moe.moe_combine_backward(c.on(c.g), c.on(c.rows), *c.route, c.w.to(DEV), c.e,
                                      grad_expand_x=out, grad_expert_scales=dw, check=True)
    dy, dw = dy.cpu(), dw.cpu()
    want = torch.full((c.cap, c.hidden), SENTINEL, dtype=torch.bfloat16)
    pairs = torch.arange(c.bs * c.k)[c.real]
    rows = (c.w.reshape(-1, 1)[pairs] * c.g.float()[pairs // c.k]).bfloat16()
    want[c.slot[pairs]] = rows
    assert torch.equal(dy, want)
    y, g = c.rows.double()[c.slot[pairs]], c.g.double()[pairs // c.k]
    dot, mag = (y * g).sum(1), (y * g).abs().sum(1)
    got = dw.double().reshape(-1)
    off = (got[pairs] - dot).abs()
    assert (off <= (c.hidden + 1) * 2.0 ** -24 * mag).all()
    assert (got[~c.real] == 0).all()
    if c.pad:
        assert (out._base[:, c.hidden:] == 77.0).all()
    return dy, dw


SHAPES = [(1, 32, 1, 1), (1, 7168, 256, 8), (5, 96, 3, 2), (33, 1056, 40, 5), (130, 64, 512, 16),
          (700, 416, 17, 3), (64, 65536, 8, 4)]


@pytest.mark.parametrize("bs,hidden,e,k", SHAPES)
def test_combine_backward(moe, bs, hidden, e, k):
    check_combine_backward(moe, Case(moe, bs, hidden, e, k, seed=bs))


@pytest.mark.parametrize("bs,hidden,e,k", [(4097, 64, 9, 1), (2049, 1056, 9, 2), (1400, 96, 17, 3),
                                           (1025, 2016, 30, 4), (900, 160, 30, 5),
                                           (601, 1024, 64, 8), (500, 64, 40, 9),
                                           (300, 32, 40, 16), (700, 480, 20, 7),
                                           (200, 768, 12, 4), (1, 512, 16, 16),
                                           (2049, 2048, 4, 2), (3, 2048, 4, 2)])
def test_combine_backward_many_short_rows(moe, bs, hidden, e, k):
    """Both sides of every change of the lanes a pair has."""
    check_combine_backward(moe, Case(moe, bs, hidden, e, k, dropped=0.2, pad=8, seed=k))
    c = Case(moe, bs, hidden, e, k, repeat=k > 1, align=1, seed=k + 1)
    dy, dw = check_combine_backward(moe, c)
    rows = c.rows.to(DEV)
    dy2, dw2 = moe.moe_combine_backward(c.g.to(DEV), rows, *c.route, c.w.to(DEV), c.e,
                                        grad_expand_x=rows)
    at = c.slot[c.real]
    assert torch.equal(dw2.cpu(), dw) and torch.equal(dy2.cpu()[at], dy[at])
    none, dw2 = moe.moe_combine_backward(c.g.to(DEV), c.rows.to(DEV), *c.route, c.w.to(DEV), c.e,
                                         need_expand_x=False)
    assert torch.equal(dw2.cpu(), dw)
    dy2, none = moe.moe_combine_backward(c.g.to(DEV), None, *c.route, c.w.to(DEV), c.e,
                                         need_scales=False, capacity_rows=c.cap)
    assert none is None and torch.equal(dy2.cpu()[at], dy[at])


@pytest.mark.parametrize("dropped", [0.3, 1.0])
def test_combine_backward_dropped_pairs(moe, dropped):
    c = Case(moe, 90, 160, 20, 4, dropped=dropped, seed=3)
    dy, dw = moe.moe_combine_backward(c.on(c.g), c.on(c.rows), *c.route, c.w.to(DEV), c.e)
    check_combine_backward(moe, c)


def test_combine_backward_repeated_ids_strides_alignments(moe):
    check_combine_backward(moe, Case(moe, 60, 224, 9, 3, repeat=True, seed=4))
    check_combine_backward(moe, Case(moe, 60, 224, 9, 3, pad=40, seed=5))
    check_combine_backward(moe, Case(moe, 60, 224, 9, 3, align=1, seed=6))


def test_combine_backward_one_output_and_in_place(moe):
    c = Case(moe, 77, 480, 30, 6, dropped=0.1, seed=7)
    dy, dw = check_combine_backward(moe, c)
    none, dw2 = moe.moe_combine_backward(c.g.to(DEV), c.rows.to(DEV), *c.route, c.w.to(DEV), c.e,
                                         need_expand_x=False)
    assert none is None and torch.equal(dw2.cpu(), dw)
    buf = torch.full((c.cap, c.hidden), SENTINEL, dtype=torch.bfloat16, device=DEV)
    dy2, none = moe.moe_combine_backward(c.g.to(DEV), None, *c.route, c.w.to(DEV), c.e,
                                         need_scales=False, grad_expand_x=buf)
    assert none is None and torch.equal(dy2.cpu(), dy)
    rows = c.rows.to(DEV)
    dy3, dw3 = moe.moe_combine_backward(c.g.to(DEV), rows, *c.route, c.w.to(DEV), c.e,
                                        grad_expand_x=rows)
    assert torch.equal(dw3.cpu(), dw)
    at = c.slot[c.real]
    assert torch.equal(dy3.cpu()[at], dy[at])
    other = torch.ones(c.cap, dtype=torch.bool)
    other[at] = False
    assert torch.equal(dy3.cpu()[other], c.rows[other])


def test_short_buffers_are_guarded(moe):
    """Rows at or beyond capacity_rows: no row, no share of a sum, flagged."""
    c = Case(moe, 50, 128, 6, 2, seed=8)
    cap = int(c.send[3]) + 2
    inside = c.slot < cap
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    buf = torch.full((c.cap, c.hidden), SENTINEL, dtype=torch.bfloat16, device=DEV)
    dy, dw = moe.moe_combine_backward(c.g.to(DEV), c.rows.to(DEV)[:cap], *c.route, c.w.to(DEV),
                                      c.e, grad_expand_x=buf[:cap], status=status)
    assert int(status.item()) == moe.MOE_FLAG_GUARD
    assert (buf[cap:] == SENTINEL).all()
    assert (dw.cpu().reshape(-1)[~inside] == 0).all()
    assert (dw.cpu().reshape(-1)[inside] != 0).all()
    status.zero_()
    dx = moe.moe_dispatch_backward(c.rows.to(DEV)[:cap], *c.route, c.e, status=status)
    assert int(status.item()) == moe.MOE_FLAG_GUARD
    want = summed(c, inside)
    assert torch.equal(dx.cpu(), want)
    none = moe.moe_dispatch_backward(c.rows.to(DEV)[:0], *c.route, c.e)
    assert (none == 0).all()


def summed(c, use, add=None):
    """fp32 sum over j ascending, then add, then one rounding."""
    s = torch.zeros((c.bs, c.hidden), dtype=torch.float32)
    use = use.reshape(c.bs, c.k)
    slot = c.slot.reshape(c.bs, c.k)
    for j in range(c.k):
        t = use[:, j].nonzero()[:, 0]
        s[t] = s[t] + c.rows.float()[slot[t, j]]
    return (s if add is None else s + add.float()).bfloat16()


@pytest.mark.parametrize("with_add", [False, True])
@pytest.mark.parametrize("bs,hidden,e,k", SHAPES)
def test_dispatch_backward(moe, bs, hidden, e, k, with_add):
    c = Case(moe, bs, hidden, e, k, seed=bs + 1)
    dx = moe.moe_dispatch_backward(c.on(c.rows), *c.route, c.e,
                                   grad_x_add=c.on(c.add) if with_add else None, check=True)
    assert torch.equal(dx.cpu(), summed(c, c.real, c.add if with_add else None))


def test_dispatch_backward_dropped_repeated_strided(moe):
    for kw in (dict(dropped=0.4), dict(dropped=1.0), dict(repeat=True), dict(pad=24),
               dict(align=1)):
        c = Case(moe, 81, 352, 11, 4, seed=12, **kw)
        for add in (None, c.add):
            dx = moe.moe_dispatch_backward(c.on(c.rows), *c.route, c.e,
                                           grad_x_add=None if add is None else c.on(add))
            assert torch.equal(dx.cpu(), summed(c, c.real, add))


def test_non_finite_values_stay_with_their_token(moe):
    c = Case(moe, 40, 128, 8, 2, seed=13)
    clean = moe.moe_dispatch_backward(c.rows.to(DEV), *c.route, c.e).cpu()
    c.rows[c.slot[2 * 7]] = float("inf")          # a row of token 7
    c.g[9] = float("nan")
    dx = moe.moe_dispatch_backward(c.rows.to(DEV), *c.route, c.e).cpu()
    assert dx[7].isinf().all()
    dy, dw = moe.moe_combine_backward(c.g.to(DEV), c.rows.to(DEV), *c.route, c.w.to(DEV), c.e)
    dy, dw = dy.cpu(), dw.cpu()
    assert dw[9].isnan().all() and dy[c.slot[18:20]].isnan().all()
    assert not dw[7, 0].isfinite()
    others = [t for t in range(40) if t not in (7, 9)]
    assert torch.equal(dx[others], clean[others]) and dw[others].isfinite().all()


# ------------------------------------------------------------------ as a trainer runs them

def forward64(c, x, y_of, w):
    """combine(experts(dispatch(x))) in 64 bits for per-expert matrices y_of."""
    rows = torch.zeros((c.cap, c.hidden), dtype=torch.float64)
    pairs = torch.arange(c.bs * c.k)[c.real]
    rows[c.slot[pairs]] = x[pairs // c.k]
    out_rows = torch.zeros_like(rows)
    for e in range(c.e):
        lo, hi = int(c.send[e]), int(c.send[e + 1])
        out_rows[lo:hi] = rows[lo:hi] @ y_of[e]
    out = torch.zeros((c.bs, c.hidden), dtype=torch.float64)
    out.index_add_(0, pairs // c.k, w.reshape(-1, 1)[pairs] * out_rows[c.slot[pairs]])
    return out, out_rows


def test_gradients_of_a_layer_against_differences(moe):
    """dispatch -> diagonal experts -> combine with loss <g, out>: the chain of
    combine_backward, the experts' own backward and dispatch_backward against
    central differences of the 64-bit forward.  The loss is linear in each of
    w and x, so a quotient has no truncation error and, in 64 bits, rounding
    far below the bounds: dw as above; dx by the bf16 roundings of w * g, of
    its product with the expert and of the sum (2^-8 each of the terms)."""
    c = Case(moe, 24, 64, 5, 3, dropped=0.1, seed=14)
    gen = torch.Generator().manual_seed(15)
    diag = torch.randn((c.e, c.hidden), generator=gen).bfloat16().double()
    y_of = torch.diag_embed(diag)
    x = torch.randn((c.bs, c.hidden), generator=gen).bfloat16()
    g = c.g.double()
    _, y64 = forward64(c, x.double(), y_of, c.w.double())
    y = y64.bfloat16()                       # what the combine read
    dy, dw = moe.moe_combine_backward(c.g.to(DEV), y.to(DEV), *c.route, c.w.to(DEV), c.e,
                                      grad_expand_x=torch.zeros((c.cap, c.hidden),
                                                                dtype=torch.bfloat16,
                                                                device=DEV))
    expert = torch.zeros((c.cap, 1), dtype=torch.int64)
    for e in range(c.e):
        expert[int(c.send[e]):int(c.send[e + 1])] = e
    d_rows = (dy.cpu().double() * diag[expert[:, 0]]).bfloat16()
    dx = moe.moe_dispatch_backward(d_rows.to(DEV), *c.route, c.e).cpu().double()
    dw = dw.cpu().double()

    def loss(x64, w64):
        return float((forward64(c, x64, y_of, w64)[0] * g).sum())

    step = 0.5
    for t, j in [(0, 0), (3, 2), (11, 1), (23, 0), (17, 2)]:
        up, down = c.w.double().clone(), c.w.double().clone()
        up[t, j] += step
        down[t, j] -= step
        q = (loss(x.double(), up) - loss(x.double(), down)) / (2 * step)
        p = t * c.k + j
        mag = float((y64[c.slot[p]] * g[t]).abs().sum()) if c.real[p] else 0.0
        # y was rounded to bf16 before the kernel read it
        assert abs(float(dw[t, j]) - q) <= (2.0 ** -8 + (c.hidden + 1) * 2.0 ** -24) * mag + 1e-9
    for t, h in [(0, 5), (7, 63), (12, 0), (20, 31), (23, 17)]:
        up, down = x.double().clone(), x.double().clone()
        up[t, h] += step
        down[t, h] -= step
        q = (loss(up, c.w.double()) - loss(down, c.w.double())) / (2 * step)
        terms = sum(abs(float(c.w[t, j] * g[t, h] * diag[c.ids[t, j].long(), h]))
                    for j in range(c.k) if c.real[t * c.k + j])
        assert abs(float(dx[t, h]) - q) <= 3.1 * 2.0 ** -8 * terms + 1e-9


def test_training_step_captured_and_replayed(moe):
    """dispatch, combine and their gradients in one graph, replayed on new
    routing and rows with eager work between: every replay equals the eager
    calls bit for bit, and two eager calls equal each other."""
    bs, hidden, e, k = 300, 512, 24, 4
    ids = torch.zeros((bs, k), dtype=torch.int32, device=DEV)
    x = torch.zeros((bs, hidden), dtype=torch.bfloat16, device=DEV)
    g = torch.zeros_like(x)
    w = torch.zeros((bs, k), device=DEV)
    cap = moe.moe_dispatch_capacity(bs, k, e)
    ws = torch.zeros(max(moe.moe_dispatch_layout_workspace_size(bs, k, e), 16),
                     dtype=torch.uint8, device=DEV)
    bufs = [torch.zeros((cap, hidden), dtype=torch.bfloat16, device=DEV) for _ in range(2)]

    def fresh(seed):
        gen = torch.Generator().manual_seed(seed)
        ids.copy_(torch.rand((bs, e), generator=gen).topk(k, 1).indices.int())
        x.copy_(torch.randn((bs, hidden), generator=gen).bfloat16())
        g.copy_(torch.randn((bs, hidden), generator=gen).bfloat16())
        w.copy_(torch.softmax(torch.randn((bs, k), generator=gen), 1))

    def step():
        for b in bufs:
            b.zero_()
        lay, ex = moe.moe_dispatch_fused(x, ids, e, expand_x=bufs[0], workspace=ws)
        r = (ids, lay.expand_idx, lay.ep_send_counts)
        out = moe.moe_combine(ex, *r, w, None, e)
        dy, dw = moe.moe_combine_backward(g, ex, *r, w, e, grad_expand_x=bufs[1])
        dx = moe.moe_dispatch_backward(dy, *r, e, grad_x_add=g)
        return out, dy, dw, dx

    fresh(0)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for seed in range(1, 5):
        fresh(seed)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in kept]
        one = [t.clone() for t in step()]
        two = [t.clone() for t in step()]
        torch.cuda.synchronize()
        for a, b, c in zip(got, one, two):
            assert torch.equal(a, b) and torch.equal(b, c)


def test_empty_batch(moe):
    ids = torch.zeros((0, 2), dtype=torch.int32, device=DEV)
    idx = torch.zeros(0, dtype=torch.int32, device=DEV)
    send = torch.zeros(5, dtype=torch.int32, device=DEV)
    rows = torch.zeros((0, 64), dtype=torch.bfloat16, device=DEV)
    w = torch.zeros((0, 2), device=DEV)
    dy, dw = moe.moe_combine_backward(rows, rows, ids, idx, send, w, 4)
    assert tuple(dy.shape) == (0, 64) and tuple(dw.shape) == (0, 2)
    assert tuple(moe.moe_dispatch_backward(rows, ids, idx, send, 4).shape) == (0, 64)
