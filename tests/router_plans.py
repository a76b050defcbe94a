"""How the weight's gradient of the router's product is made at given sizes, by
the library's rule as it stands, written again from its comments: in ranges of
tokens from grad_logits as they are, or by tiles from parts of them that are
made beforehand, in shares of the tokens.  The workspace's size tells the two
apart, and the numbers of ranges and shares, so the rule here is checked
against the library (test_router_plans.py) and the tests that need one way or
the other ask for it by this."""

from typing import NamedTuple

import numpy as np

f32 = np.float32
UNITS, DEPTH = 256, 64


def ceil_div(n, by):
    return -(-n // by)


class Plan(NamedTuple):
    ranges: int        # of tokens, 0: by parts
    tile: tuple        # channels x experts of a tile (by parts)
    shares: int        # of the tokens (by parts)


# (channels, experts, workgroups a unit, us of the ends, of a block, of a block where
# two share a unit)
TILES = [(64, 64, 2, 3.0, 0.75, 0.85), (256, 128, 1, 4.0, 2.4, 2.4)]


def by_parts(bs, h, e):
    """(us, tile, shares) of the cheapest tile and number of shares."""
    best = (f32(3e38), None, 0)
    blocks = ceil_div(bs, DEPTH)
    for ti, tj, a_unit, ends, block, of_two in TILES:
        tiles = ceil_div(h, ti) * ceil_div(e, tj)
        for shares in range(1, min(32, blocks) + 1):
            jobs, places = tiles * shares, a_unit * UNITS
            if shares > 1 and jobs > 2 * places:
                break
            each = f32(of_two if jobs > UNITS else block)
            us = f32(ceil_div(jobs, places)) * (f32(ends) + each * f32(ceil_div(blocks, shares)))
            if shares > 1:
                us += f32(2) + f32(shares) * f32(h) * f32(e) * f32(1e-6)
            if us < best[0]:
                best = (us, (ti, tj), shares)
    return best


def plan(bs, h, e) -> Plan:
    us, tile, shares = by_parts(bs, h, e)
    stages, tiles = ceil_div(bs, DEPTH), ceil_div(h, 128) * ceil_div(e, 64)
    least, best = us + f32(9), 0
    for r in range(1, min(stages, 96) + 1):
        jobs = tiles * r
        cost = f32(ceil_div(jobs, UNITS)) * (f32(2) + f32(1.6) * f32(ceil_div(stages, r)))
        if jobs > UNITS // 2:
            cost += f32(2.5)
        if r > 1:
            cost += f32(2.5) + f32(r) * (f32(0.03) + f32(e) * f32(h) * f32(1e-6))
        if cost < least:
            least, best = cost, r
    return Plan(best, None, 0) if best else Plan(0, tile, shares)


def workspace_bytes(bs, h, e):
    """What the gradient asks for by that plan."""
    p = plan(bs, h, e)
    if p.ranges:
        return 0 if p.ranges == 1 else p.ranges * e * h * 4
    parts = 3 * 2 * DEPTH * ceil_div(bs, DEPTH) * DEPTH * ceil_div(e, DEPTH)
    return parts + (0 if p.shares == 1 else p.shares * e * h * 4)


# Sizes that go by parts, each tile with one share and several.
BY_PARTS = [(164, 5408, 351, (64, 64), 1), (321, 5760, 343, (64, 64), 1),
            (3000, 1056, 512, (64, 64), 3), (2881, 2080, 130, (64, 64), 5),
            (70, 16384, 300, (256, 128), 1), (465, 5760, 343, (256, 128), 3),
            (2673, 4192, 74, (256, 128), 14)]
# Tokens up to which a size goes one way (ranges or parts), and the first to parts of
# another tile.
CHANGES = [(4608, 2048, 128), (2880, 2080, 130), (128, 5408, 351), (320, 5760, 343),
           (448, 5760, 343)]
