"""The rule that chooses an experts' product's tile, on the CPU: the sizes
that the GPU tests run are on both sides of every change, and reach every
tile."""

import pytest

import combine_moe_dispatch_layout_amd as moe
import product_tiles as sizes


def tile(s, expected_rows, gated, grouped=True, rows=None):
    return moe.moe_probe_product_tile(s["rows"] if rows is None else rows, s["experts"], s["out"],
                                      expected_rows=expected_rows, gated=gated, grouped=grouped)


@pytest.mark.parametrize("name,gated,grouped", [("GATED", True, True), ("PLAIN_FEW", False, True),
                                                ("PLAIN_MANY", False, True),
                                                ("DENSE", False, False)])
def test_tiles_of_the_listed_sizes(name, gated, grouped):
    s = getattr(sizes, name)
    got = {r: tile(s, r, gated, grouped) for r, _ in s["cases"]}
    assert got == dict(s["cases"])
    # every change between the least and the most rows has its two sides listed
    rows = [r for r, _ in s["cases"]]
    changes = [r for r in range(rows[0] + 1, rows[-1] + 1)
               if tile(s, r, gated, grouped) != tile(s, r - 1, gated, grouped)]
    assert all(r in got and r - 1 in got for r in changes)
    # unknown rows, or more than fit: as many as fit
    for r in (0, s["rows"], 10 ** 9):
        assert tile(s, r, gated, grouped) == tile(s, s["rows"], gated, grouped)


def test_every_tile_is_reached():
    assert {t for _, t in sizes.GATED["cases"]} == sizes.GATED_TILES
    plain = sizes.PLAIN_FEW["cases"] + sizes.PLAIN_MANY["cases"]
    assert {t for _, t in plain} == sizes.PLAIN_TILES
    # and no call takes another
    for experts in (1, 2, 7, 32, 256, 512):
        for out in (128, 1408, 7168, 32768):
            for rows in (1, 7, 16, 20, 33, 48, 64, 96, 97, 128, 500, 5000):
                for gated, tiles in ((False, sizes.PLAIN_TILES), (True, sizes.GATED_TILES)):
                    assert moe.moe_probe_product_tile(rows * experts, experts, out,
                                                      gated=gated) in tiles


@pytest.mark.parametrize("kw", [
    dict(capacity_rows=0), dict(capacity_rows=-1), dict(capacity_rows=(1 << 30) + 1),
    dict(num_experts=0), dict(num_experts=513), dict(out_features=0), dict(out_features=8),
    dict(out_features=65568), dict(expected_rows=-1), dict(grouped=False),
    dict(gated=True, out_features=160), dict(gated=True, out_features=32896),
])
def test_sizes_that_the_product_refuses(kw):
    a = dict(capacity_rows=100, num_experts=4, out_features=256)
    a.update(kw)
    with pytest.raises(moe.MoeError):
        moe.moe_probe_product_tile(a.pop("capacity_rows"), a.pop("num_experts"),
                                   a.pop("out_features"), **a)
    lib = moe.load_library()
    assert lib.moe_probe_product_tile(0, 1, 100, 4, 256, 0, None, None, None) == 1
