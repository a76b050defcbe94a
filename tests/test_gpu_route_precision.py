"""The routing's weights and gradients are those of 64-bit scores, rounded once.

Bars, from the arithmetic alone: a weight is a quotient of 64-bit exponentials
and sums, off by 2^-28 of itself with room to spare, and rounded to fp32, which
is off by 2^-24 at most.  A gradient's factors likewise, the first of them of the
terms' magnitudes (what is taken off may cancel).  A softmax over all experts
divides by a sum of fp32 exponentials: 2^-19 of itself."""

import numpy as np
import pytest
import torch

import router_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
ONCE = 2.0 ** -24
INSIDE = 2.0 ** -28
SUM = 2.0 ** -19


@pytest.fixture(scope="module")
def moe():
    import combine_moe_dispatch_layout_amd as m
    m.load_library()
    assert torch.cuda.is_available()
    return m


def by_formula(grad, logits, ids, score, renormalize, scale):
    """(gradient, magnitude of its terms).  router_reference's, but that a sigmoid's
    1 - s is 1 / (1 + e^l): taken from 1, a score near 1 leaves nothing of 64 bits."""
    if score == "softmax":
        return ref.route_backward(grad, logits, ids, score, renormalize, scale)
    l, s = ref.scores(logits.astype(np.float64), score)
    q, g = ref.weights(s, ids, renormalize), np.where(ids >= 0, grad.astype(np.float64), 0.0)
    with np.errstate(over="ignore"):
        rest = 1 / (1 + np.exp(np.take_along_axis(l, np.maximum(ids, 0), 1)))
    dot = (g * q).sum(1, keepdims=True) if renormalize else 0.0
    mag = np.abs(g * q).sum(1, keepdims=True) if renormalize else 0.0
    want, size = np.zeros_like(l), np.zeros_like(l)
    rows = np.arange(len(l))
    for j in range(ids.shape[1]):
        at = np.maximum(ids[:, j], 0)
        want[rows, at] += (q * rest * (g - dot))[:, j] * (ids[:, j] >= 0)
        size[rows, at] += (q * rest * (np.abs(g) + mag))[:, j] * (ids[:, j] >= 0)
    return scale * want, scale * size


# Logits near 0, of the usual size, and so far apart that scores leave fp32.
@pytest.mark.parametrize("spread", [0.1, 3.0, 30.0])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bs,e,k", [(300, 60, 6), (100, 256, 16), (2600, 512, 8), (6200, 130, 9)])
def test_weights_and_gradients(moe, bs, e, k, score, renormalize, spread):
    gen = torch.Generator().manual_seed(bs + e)
    l = spread * torch.randn((bs, e), generator=gen)
    l[::5] -= 3 * spread
    bias = None if e == 60 else 0.1 * torch.randn(e, generator=gen)
    if bias is None:
        l[1::7, ::3] = float("-inf")
    ld = l.to(DEV)
    kw = dict(score=score, renormalize=renormalize, scale=2.5)
    ids, w = moe.moe_route(ld, k, bias=None if bias is None else bias.to(DEV), **kw)
    _, want = ref.route(l.numpy(), k, bias=None if bias is None else bias.numpy(), **kw)
    inside = SUM if score == "softmax" and not renormalize else INSIDE
    err = np.abs(w.cpu().double().numpy() - want)
    least = 2.0 ** -149     # fp32's smallest step
    assert (err <= (ONCE + inside) * np.abs(want) + least).all()
    g = torch.randn((bs, k), generator=gen)
    d = moe.moe_route_backward(g.to(DEV), ld, ids, **kw).cpu().double().numpy()
    want, size = by_formula(g.numpy(), l.numpy(), ids.cpu().numpy(), **kw)
    if inside == INSIDE:
        assert (np.abs(d - want) <= ONCE * np.abs(want) + INSIDE * size + least).all()
    else:
        # Every expert's fp32 exponential of a rounded difference, too.  Where that
        # leaves the normal numbers it is off by half of 2^-149, and so is what becomes
        # of it times scale * dot / sum, which is below 2.5 * sum |g|, and its product.
        every = ref.score_error(l.numpy()) + 2 * SUM
        least = least * (1 + 2.5 * np.abs(g.numpy()).sum(1, keepdims=True))
        assert (np.abs(d - want) <= ONCE * np.abs(want) + every * size + least).all()
