"""The weight's gradient of the router's product from parts of grad_logits that
are made beforehand: all 24 bits of them arrive, in every tile, with and
without shares of the tokens.  Each size's way is checked on the CPU
(test_router_plans.py).

Bars: what is compared bit for bit has sums that are exact in any order (one
term each, or whole numbers whose magnitudes add up to less than 2^24); the
others are router_reference's kind, an fp32 sum of n terms by (n + 64) units of
2^-23 of their summed magnitude for each of three parts."""

import pytest
import torch

import router_plans as plans

pytestmark = pytest.mark.gpu

DEV = "cuda"
SIZES = [s[:3] for s in plans.BY_PARTS]


@pytest.fixture(scope="module")
def moe():
    import combine_moe_dispatch_layout_amd as m
    m.load_library()
    assert torch.cuda.is_available()
    return m


def grad_weight(moe, g, x, e, **kw):
    w = torch.zeros((e, x.shape[1]), dtype=torch.bfloat16, device=DEV)
    return moe.moe_router_logits_backward(g.to(DEV), x.to(DEV), w, **kw)[1].cpu()


@pytest.mark.parametrize("bs,h,e", SIZES)
def test_every_bit(moe, bs, h, e):
    """One token in each channel: the gradient is grad_logits themselves, down
    to 2^-133, the smallest step that a bf16 part has.  (The parts' last is rounded
    to that step, so what is below 2^-110, whose 24th bit lies under it, may be off by
    half of it, 2^-134; above, half of that step is less than a bit, and the values are
    equal.)"""
    gen = torch.Generator().manual_seed(bs)
    g = torch.randn((bs, e), generator=gen)
    g = g * torch.pow(2.0, torch.randint(-100, 120, (bs, e), generator=gen).float())
    token = torch.randint(0, bs, (h,), generator=gen)
    token[:2], token[-2:] = bs - 1, 0
    x = torch.zeros((bs, h))
    x[token, torch.arange(h)] = 1.0
    want = g[token].t()
    for kw in (dict(), dict(need_x=False)):
        dw = grad_weight(moe, g, x.bfloat16(), e, **kw)
        assert ((dw.double() - want.double()).abs() <= 2.0 ** -134).all()


@pytest.mark.parametrize("bs,h,e", SIZES)
def test_sums_of_whole_numbers_that_need_three_parts(moe, bs, h, e):
    """Eight tokens a channel, of odd numbers of up to 21 bits."""
    gen = torch.Generator().manual_seed(bs + 1)
    g = 2 * torch.randint(-(1 << 20), 1 << 20, (bs, e), generator=gen).float() + 1
    x = torch.zeros((bs, h), dtype=torch.float64)
    for n in range(8):
        token = torch.randint(0, bs, (h,), generator=gen)
        x[token, torch.arange(h)] = 1.0 if n % 3 else -1.0
    want = g.double().t() @ x
    assert want.abs().max() < 1 << 24
    assert torch.equal(grad_weight(moe, g, x.bfloat16(), e).double(), want)


@pytest.mark.parametrize("bs,h,e", SIZES)
def test_non_finite_values(moe, bs, h, e):
    x = torch.ones((bs, h), dtype=torch.bfloat16)
    g = torch.ones((bs, e))
    g[2, 3], g[bs - 1, 5] = float("inf"), float("-inf")
    g[9, 4] = float("nan")
    g[5, 6] = 3.3e38
    loud = torch.tensor([0x7F800001, -0x7FFFFF], dtype=torch.int32).view(torch.float32)
    g[11, 7], g[bs - 2, 8] = loud[0], loud[1]    # their marks lie in the lowest bits
    dw = grad_weight(moe, g, x, e)
    assert (dw[3] == float("inf")).all() and (dw[5] == float("-inf")).all()
    assert dw[[4, 7, 8]].isnan().all() and dw[6].isfinite().all()
    rest = [i for i in range(e) if i not in (3, 4, 5, 6, 7, 8)]
    assert (dw[rest] == bs).all()
    x[bs - 1, 7] = float("inf")     # next to what pads the last stage
    x[0, h - 1] = float("nan")
    dw = grad_weight(moe, torch.zeros((bs, e)), x, e)
    assert dw[:, [7, h - 1]].isnan().all()
    dw[:, [7, h - 1]] = 0
    assert (dw == 0).all()


def on(t, pad):
    buf = torch.full((t.shape[0], t.shape[1] + pad), 55.0, device=DEV)
    buf[:, :t.shape[1]] = t.to(DEV)
    return buf[:, :t.shape[1]]


@pytest.mark.parametrize("bs,h,e", sorted({(bs + more, h, e) for bs, h, e in plans.CHANGES
                                           for more in (0, 1)}))
def test_both_sides_of_each_change(moe, bs, h, e):
    """Rows of grad_logits that begin at 16 bytes or not, and the gradients asked
    for one by one: the same bits."""
    gen = torch.Generator().manual_seed(bs + h)
    x = torch.randn((bs, h), generator=gen).bfloat16().to(DEV)
    w = torch.randn((e, h), generator=gen).bfloat16().to(DEV)
    g = torch.randn((bs, e), generator=gen)
    dx, dw = moe.moe_router_logits_backward(g.to(DEV), x, w)
    g64, x64 = g.double(), x.cpu().double()
    bound = (2.0 ** -24 + 3 * (bs + 64) * 2.0 ** -23) * (g64.abs().t() @ x64.abs())
    assert ((dw.cpu().double() - g64.t() @ x64).abs() <= bound).all()
    for pad in (1, 4):
        dx2, dw2 = moe.moe_router_logits_backward(on(g, pad), x, w)
        assert torch.equal(dx2, dx) and torch.equal(dw2, dw)
    odd = torch.zeros(bs * e + 1, device=DEV)[1:].view(bs, e)
    odd.copy_(g)
    assert torch.equal(moe.moe_router_logits_backward(odd, x, w, need_x=False)[1], dw)
    assert torch.equal(moe.moe_router_logits_backward(odd, x, w, need_weight=False)[0], dx)


@pytest.mark.parametrize("bs,h,e", [(20, 96, 24), (300, 96, 24), *SIZES[2:3]])
def test_infinite_rows_and_weights_spoil_what_they_enter_alone(moe, bs, h, e):
    """An infinity in x or weight gives an infinity or a NaN, and nothing else."""
    x, g = torch.ones((bs, h)), torch.ones((bs, e))
    w = torch.ones((e, h))
    x[3, 5], w[2, 7] = float("inf"), float("-inf")
    g[3, 0] = 1.7e-3     # three parts
    dx, dw = moe.moe_router_logits_backward(g.to(DEV), x.bfloat16().to(DEV), w.bfloat16().to(DEV))
    dx, dw = dx.cpu().float(), dw.cpu()
    assert not dw[:, 5].isfinite().any() and not dx[:, 7].isfinite().any()
    dw[:, 5], dx[:, 7] = bs, e
    assert (dw[1:] == bs).all() and (dx[[0, 1, 2, 4]] == e).all()


@pytest.mark.parametrize("bs,h,e", [(1, 64, 8), (40, 256, 60), (5000, 256, 60), (4200, 512, 256),
                                    (2000, 512, 512)])
def test_terms_of_the_rows_gradient_that_cancel(moe, bs, h, e):
    """Pairs of experts with one weight and all but opposite gradients: what is
    lost is held to 2^-16 of the terms' magnitudes and the fp32 sums' rounding."""
    gen = torch.Generator().manual_seed(bs + e)
    w = torch.randn((e // 2, h), generator=gen).bfloat16().repeat_interleave(2, 0)
    g = torch.randn((bs, e // 2), generator=gen).repeat_interleave(2, 1)
    g[:, 1::2] *= -(1 - 2.0 ** -18)
    x = torch.zeros((bs, h), dtype=torch.bfloat16, device=DEV)
    dx, _ = moe.moe_router_logits_backward(g.to(DEV), x, w.to(DEV), need_weight=False)
    want = g.double() @ w.double()
    mag = g.double().abs() @ w.double().abs()
    bound = 2.0 ** -8 * want.abs() + 1.01 * (2.0 ** -16 + (2 * e + 64) * 2.0 ** -23) * mag
    assert ((dx.cpu().double() - want).abs() <= bound).all()
