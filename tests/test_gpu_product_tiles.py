"""The experts' products in every tile they have, on the GPU: on both sides
of every change of tile, with sums that begin at the first block and with ones
that begin at a block of their column's own (4096 channels), and with rows at
the longest stride.  Which tile a call takes is asked of the library, so a
later change of the rule cannot empty these tests.

Bars: where every sum is exact the outputs equal the rounded 64-bit ones bit
for bit; with general values the first call is within half a bf16 (or e4m3)
step and the sums' bound, and every other equals it bit for bit.  The 64-bit
products run on the GPU, an expert at a time."""

import math

import numpy as np
import pytest
import torch

import experts_reference as ref
import product_tiles as sizes
from test_gpu_experts import gated_reference

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def moe():
    import combine_moe_dispatch_layout_amd as m
    m.load_library()
    assert torch.cuda.is_available()
    return m


def counts_of(experts, rows):
    """Rows of each expert, all of `rows` but two: none, one, both sides of
    tile edges, and the rest."""
    some = [0, 1, 32, 33, 63, 64, 65, 128, 129, 31, 96, 97, 255, 257]
    if experts == 1:
        return [rows]
    if experts == 2:
        return [rows - 2 - 385, 385]
    counts = some + [1] * (experts - 1 - len(some))
    while sum(counts) > rows - 200:      # leave a long one for the last
        counts[counts.index(max(counts))] //= 2
    return counts + [rows - 2 - sum(counts)]


class Inputs:
    """One set of sizes' rows and weights; rows of no expert lie behind the
    last and between two of them."""

    def __init__(self, s, channels, gated, exact, seed):
        gen = torch.Generator().manual_seed(seed)
        e, self.cap = s["experts"], s["rows"]
        self.n = s["out"] * (2 if gated else 1)
        self.counts = counts_of(e, self.cap)
        self.send = np.concatenate([[0], np.cumsum(self.counts)]).astype(np.int32)
        if e > 1:
            self.send[e // 2:] += 1
        codes = ref.small_codes if exact else ref.random_codes
        scales = ref.power_scales if exact else ref.random_scales
        self.real = ref.real_rows(self.cap, self.counts, self.send)
        x = codes(gen, (self.cap, channels))
        x[~self.real] = 0x7F
        xs = scales(gen, (self.cap, channels // 128))
        xs[~self.real] = float("nan")
        w = codes(gen, (1, self.n, channels)).to(DEV).repeat(e, 1, 1)
        for i in range(1, e):            # other weights for each expert
            w[i] = w[0].roll(37 * i, 0).roll(128 * i, 1)
        ws = scales(gen, (e, -(-self.n // 128), channels // 128))
        if not exact:
            ws *= 0.02 / math.sqrt(channels)
        self.x, self.xs, self.w, self.ws = x.to(DEV), xs.to(DEV), w, ws.to(DEV)
        self.meta = (torch.tensor(self.counts, dtype=torch.int32, device=DEV),
                     torch.from_numpy(self.send).to(DEV)) if e > 1 else (None, None)

    def args(self, x=None):
        return (self.x if x is None else x, self.xs, self.w, self.ws, *self.meta)

    def product(self):
        """(y, summed magnitudes), on the CPU."""
        f64 = torch.float64
        value = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).to(f64).to(DEV)
        y = torch.zeros((self.cap, self.n), dtype=f64, device=DEV)
        mag = torch.zeros_like(y)
        for i, c in enumerate(self.counts):
            lo = int(self.send[i])
            a = value[self.x[lo:lo + c].long()]
            a *= self.xs[lo:lo + c].to(f64).repeat_interleave(128, 1)
            w = value[self.w[i].long()] * self.ws[i].to(f64).repeat_interleave(
                128, 0)[:self.n].repeat_interleave(128, 1)
            wt = w.t().contiguous()
            y[lo:lo + c] = a @ wt
            mag[lo:lo + c] = a.abs() @ wt.abs()
        return y.cpu(), mag.cpu()


SETS = [("PLAIN_FEW", True), ("PLAIN_MANY", True), ("DENSE", False)]


def plain_run(moe, inp, s, grouped, expected_rows, want_tile, x=None):
    tile = moe.moe_probe_product_tile(inp.cap, s["experts"], inp.n, expected_rows=expected_rows,
                                      grouped=grouped)
    assert tile == want_tile
    out = torch.full((inp.cap, inp.n), ref.SENTINEL_OUT, dtype=torch.bfloat16, device=DEV)
    moe.moe_grouped_gemm_fp8(*inp.args(x), out=out, expected_rows=expected_rows, check=True)
    return out.cpu()


@pytest.mark.parametrize("channels", [384, 4096])
@pytest.mark.parametrize("name,grouped", SETS)
def test_plain_tiles_exact(moe, name, grouped, channels):
    s = getattr(sizes, name)
    inp = Inputs(s, channels, False, True, seed=channels)
    want = inp.product()[0].bfloat16()
    want[~inp.real] = ref.SENTINEL_OUT
    for r, tile in s["cases"]:
        assert torch.equal(plain_run(moe, inp, s, grouped, r, tile), want), (r, tile)


@pytest.mark.parametrize("channels", [384, 4096])
@pytest.mark.parametrize("name,grouped", SETS)
def test_plain_tiles_general_values(moe, name, grouped, channels):
    s = getattr(sizes, name)
    inp = Inputs(s, channels, False, False, seed=channels + 1)
    y, mag = inp.product()
    first = None
    for r, tile in s["cases"]:
        out = plain_run(moe, inp, s, grouped, r, tile)
        if first is None:
            first = out
            bound = 2.0 ** -8 * y.abs() + (1 + 2.0 ** -8) * ref.e4m3_sum_error(channels) * mag
            assert ((out.double() - y).abs() <= bound)[inp.real].all()
            assert (out[~inp.real] == ref.SENTINEL_OUT).all()
        assert torch.equal(out.view(torch.int16), first.view(torch.int16)), (r, tile)


def far_rows(inp, channels):
    """The rows 2^23 bytes apart."""
    far = torch.empty((inp.cap, 1 << 23), dtype=torch.uint8, device=DEV)[:, :channels]
    far.copy_(inp.x)
    return far


@pytest.mark.parametrize("name,grouped", SETS)
def test_plain_tiles_longest_row_stride(moe, name, grouped):
    s = getattr(sizes, name)
    inp = Inputs(s, 256, False, True, seed=3)
    want = inp.product()[0].bfloat16()
    want[~inp.real] = ref.SENTINEL_OUT
    far = far_rows(inp, 256)
    for r, tile in s["cases"]:
        assert torch.equal(plain_run(moe, inp, s, grouped, r, tile, far), want), (r, tile)


def gated_run(moe, inp, s, expected_rows, want_tile, x=None):
    tile = moe.moe_probe_product_tile(inp.cap, s["experts"], inp.n // 2,
                                      expected_rows=expected_rows, gated=True)
    assert tile == want_tile
    inter = inp.n // 2
    out = torch.full((inp.cap, inter), ref.SENTINEL_CODE, dtype=torch.uint8, device=DEV)
    scales = torch.full((inp.cap, inter // 128), ref.SENTINEL_SCALE, device=DEV)
    moe.moe_grouped_gemm_silu_fp8(*inp.args(x), out=out, out_scales=scales,
                                  expected_rows=expected_rows, check=True)
    return out.cpu(), scales.cpu()


@pytest.mark.parametrize("channels,far", [(384, False), (4096, False), (256, True)])
def test_gated_tiles(moe, channels, far):
    s = sizes.GATED
    inp = Inputs(s, channels, True, False, seed=channels + 2)
    h, dh = gated_reference(*inp.product(), channels)
    x = far_rows(inp, channels) if far else None
    first = None
    for r, tile in s["cases"]:
        codes, scales = gated_run(moe, inp, s, r, tile, x)
        if first is None:
            first = codes, scales
            real = inp.real
            blocks = h.view(h.shape[0], -1, 128)
            want = blocks.abs().amax(2) / 448
            ds = dh.view(blocks.shape).amax(2) / 448 + 2.0 ** -23 * want
            assert ((scales.double() - want).abs() <= ds)[real].all()
            wide = scales.double().repeat_interleave(128, 1)
            # half an e4m3 step, and what h and the scale are off by
            bound = 2.0 ** -4 * h.abs() + 2.0 ** -10 * wide + 1.1 * dh \
                + 448 * ds.repeat_interleave(128, 1)
            assert ((ref.values(codes) * wide - h).abs() <= bound)[real].all()
            assert (codes[~real] == ref.SENTINEL_CODE).all()
            assert (scales[~real] == ref.SENTINEL_SCALE).all()
        assert torch.equal(codes, first[0]) and torch.equal(scales, first[1]), (r, tile)
