"""The weight's gradient of the router's product: the rule that router_plans
writes down is the library's, by the workspace that each way asks for."""

import random

import pytest

import combine_moe_dispatch_layout_amd as moe
import router_plans as plans


@pytest.mark.parametrize("seed", range(4))
def test_the_rule_is_the_librarys(seed):
    rng = random.Random(seed)
    for _ in range(3000):
        bs = int(2 ** rng.uniform(0, 15))
        h = 32 * int(2 ** rng.uniform(0, 10))
        e = rng.randint(1, 512)
        assert plans.workspace_bytes(bs, h, e) == \
            moe.moe_router_logits_backward_workspace_size(bs, h, e), (bs, h, e)


@pytest.mark.parametrize("bs,h,e,tile,shares", plans.BY_PARTS)
def test_sizes_by_parts(bs, h, e, tile, shares):
    assert plans.plan(bs, h, e) == (0, tile, shares)


def test_sizes_by_parts_have_every_tile_with_and_without_shares():
    assert {(tile, shares > 1) for *_, tile, shares in plans.BY_PARTS} == {
        (tile[:2], more) for tile in plans.TILES for more in (False, True)}


@pytest.mark.parametrize("bs,h,e", plans.CHANGES)
def test_changes(bs, h, e):
    """One token more goes another way."""
    here, there = plans.plan(bs, h, e), plans.plan(bs + 1, h, e)
    assert (here.ranges == 0, here.tile) != (there.ranges == 0, there.tile)
