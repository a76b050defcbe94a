"""Groups whose scores are sums that cancel: the choice is that of 64-bit keys,
whatever fp32 makes of keys that are far larger than their sum."""

import numpy as np
import pytest
import torch

import router_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def moe():
    import combine_moe_dispatch_layout_amd as m
    m.load_library()
    assert torch.cuda.is_available()
    return m


def check(moe, l, bias, k, **kw):
    ids, _ = moe.moe_route(l.to(DEV), k, bias=bias.to(DEV), **kw)
    want, _ = ref.route(l.float().numpy(), k, bias=bias.numpy(), **kw)
    assert np.array_equal(ids.cpu().numpy(), want)


def test_two_rows_that_fp32_decides_wrongly(moe):
    """Sigmoid: group 0 has 1.0827974, group 1 1.0827995, and in fp32 1.0828247
    and 1.0827994.  Softmax: 2^-9 each, group 1 is ahead by 6e-8, in fp32 behind."""
    l = torch.tensor([[1.3706665, -0.9182745, -1.0656360, 1.5614803]])
    bias = torch.tensor([1000.0, -1000.0, 0.1, -0.1])
    check(moe, l, bias, 1, score="sigmoid", groups=2, top_groups=1)
    u = 2.0 ** -24
    v = round(0.99 / u) * u
    bias = torch.full((512,), -4.0)
    bias[0], bias[1] = 1 - 2.0 ** -9 + 3 * u, -v - 2.0 ** -9
    bias[256], bias[257] = 1 - 2.0 ** -9 + 5 * u, -v - 2.0 ** -9 - u
    check(moe, torch.zeros((3, 512)), bias, 2, score="softmax", groups=2, top_groups=1)


def bias_of_both_signs(gen, e, groups, size):
    """Each group's two best keys are near size and -size, the others lower."""
    bias = torch.full((e,), -4.0 * size)
    of = e // groups
    for g in range(groups):
        bias[g * of] = size + 0.1 * torch.randn(1, generator=gen)
        bias[g * of + 1] = -size + 0.1 * torch.randn(1, generator=gen)
    return bias


# A wave and 16 lanes a row, groups of several lanes, a lane and more than lanes.
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [1.0, 30.0, 1000.0, 1e5])
@pytest.mark.parametrize("bs,e,groups,top", [(300, 4, 2, 1), (4100, 64, 8, 3), (1000, 256, 8, 4),
                                             (4100, 256, 8, 4), (4100, 512, 64, 9),
                                             (2000, 128, 64, 9), (4100, 500, 5, 2)])
def test_groups_of_keys_of_both_signs(moe, bs, e, groups, top, size, score):
    gen = torch.Generator().manual_seed(bs + e + groups)
    bias = bias_of_both_signs(gen, e, groups, size)
    l = 2 * torch.randn((bs, e), generator=gen)
    l[1::9, e // groups:] = float("-inf")     # one group is left
    l[2::9] = l[2::9].masked_fill(torch.rand((len(l[2::9]), e), generator=gen) < 0.3,
                                  float("-inf"))
    for group_score in ("top2", "max"):
        check(moe, l, bias, min(6, 2 * top), score=score, groups=groups, top_groups=top,
              group_score=group_score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bs", [200, 4200])
def test_group_scores_that_leave_fp32(moe, score, bs):
    """Sums past fp32's largest and biases of infinity go by 64 bits."""
    gen = torch.Generator().manual_seed(bs)
    l = torch.randn((bs, 64), generator=gen)
    bias = torch.randn(64, generator=gen)
    for at, value in ((0, 3e38), (1, 2e38), (8, 3e38), (9, 3e38), (17, -3e38), (24, 3.3e38)):
        bias[at] = value
    check(moe, l, bias, 4, score=score, groups=8, top_groups=2)
    bias[40] = float("inf")
    check(moe, l, bias, 4, score=score, groups=8, top_groups=3)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bs,e,k,groups,top", [(128, 256, 8, 8, 4), (4100, 512, 16, 16, 3),
                                               (4099, 128, 5, 64, 9), (300, 60, 6, 6, 3)])
def test_bf16_logits(moe, bs, e, k, groups, top, score):
    """Logits of 8 bits: many keys and groups are equal, and go to the lowest."""
    gen = torch.Generator().manual_seed(bs + e)
    l = torch.randn((bs, e), generator=gen).bfloat16()
    l[1::3] = (2 * l[1::3]).round() / 2
    l[2::5] = l[2::5].masked_fill(torch.rand((len(l[2::5]), e), generator=gen) < 0.6,
                                  float("-inf"))
    few = 0.25 * torch.randint(-2, 3, (e,), generator=gen).float()
    for group_score in ("top2", "max"):
        for bias in (torch.zeros(e), few, 0.1 * torch.randn(e, generator=gen)):
            check(moe, l, bias, k, score=score, groups=groups, top_groups=top,
                  group_score=group_score)
        ids, _ = moe.moe_route(l.to(DEV), k, score=score, groups=groups, top_groups=top,
                               group_score=group_score)
        want, _ = ref.route(l.float().numpy(), k, score=score, groups=groups, top_groups=top,
                            group_score=group_score)
        assert np.array_equal(ids.cpu().numpy(), want)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [3.3, 30.0, 1000.0, 1e5])
@pytest.mark.parametrize("bs,e,k", [(300, 24, 16), (4200, 64, 12), (500, 256, 16),
                                    (4200, 512, 16)])
def test_experts_far_below_the_best(moe, bs, e, k, size, score):
    """Keys of another size than the largest one's, nearer to each other than
    their own roundings."""
    gen = torch.Generator().manual_seed(bs + e)
    l = torch.randn((bs, e), generator=gen)
    for most, rest in ((0.0, -size), (size, 0.0), (size, -size)):
        bias = rest + 1e-7 * size * torch.randn(e, generator=gen)
        bias[::7] = most + 0.1 * torch.randn(len(bias[::7]), generator=gen)
        check(moe, l, bias, k, score=score)
