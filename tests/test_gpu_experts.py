"""The experts' products on the GPU against plain 64-bit forms.

Bars, from the arithmetic alone: where every product, scale and sum is
exact the bf16 output must equal the rounded 64-bit result bit for bit; with
general values the error is at most half a bf16 step (2^-8 of the value) plus
the sums' bound (experts_reference.e4m3_sum_error).  The gated form's
dequantised output is within half an e4m3 step of the 64-bit h (2^-4 of the
value, or half the smallest step, 2^-10 of the scale) plus the propagated
error of the sums.  Rows of no expert keep what they held.
"""

import math

import numpy as np
import pytest
import torch

import experts_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def moe():
    import combine_moe_dispatch_layout_amd as m
    m.load_library()
    assert torch.cuda.is_available()
    return m


def padded_rows(t, pad):
    """t [R, C] on the GPU as a view of rows `pad` elements longer."""
    buf = torch.zeros((t.shape[0], t.shape[1] + pad), dtype=t.dtype, device=DEV)
    buf[:, :t.shape[1]] = t.to(DEV)
    return buf[:, :t.shape[1]]


class Inputs:
    def __init__(self, counts, n, channels, *, align=128, extra=0, exact=False, seed=0, pad=0):
        gen = torch.Generator().manual_seed(seed)
        self.counts = counts
        self.send = ref.segments(counts, align)
        self.cap = int(self.send[-1]) + extra
        e = len(counts)
        codes = ref.small_codes if exact else ref.random_codes
        scales = ref.power_scales if exact else ref.random_scales
        self.x = codes(gen, (self.cap, channels))
        self.xs = scales(gen, (self.cap, channels // 128))
        self.w = codes(gen, (e, n, channels))
        self.ws = scales(gen, (e, -(-n // 128), channels // 128))
        if not exact:
            # like a real layer's, so that the gate stays in silu's range
            self.ws *= 0.02 / math.sqrt(channels)
        self.real = ref.real_rows(self.cap, counts, self.send)
        # what lies in rows of no expert must not matter
        self.x[~self.real] = 0x7F
        self.xs[~self.real] = float("nan")
        self.gpu = (padded_rows(self.x, pad), self.xs.to(DEV), self.w.to(DEV), self.ws.to(DEV),
                    torch.tensor(counts, dtype=torch.int32, device=DEV),
                    torch.from_numpy(self.send).to(DEV))

    def product(self):
        x = ref.dequantised(self.x, self.xs)
        x[~self.real] = 0
        return ref.product(x, ref.weight_values(self.w, self.ws), self.counts, self.send)


def check_product(moe, inp, exact, expected_rows=None, pad=0):
    n = inp.w.shape[1]
    buf = torch.full((inp.cap, n + pad), ref.SENTINEL_OUT, dtype=torch.bfloat16, device=DEV)
    out = moe.moe_grouped_gemm_fp8(*inp.gpu, out=buf[:, :n], expected_rows=expected_rows,
                                   check=True)
    torch.cuda.synchronize()
    got = out.cpu()
    y, mag = inp.product()
    if exact:
        assert torch.equal(got[inp.real], y[inp.real].bfloat16())
    else:
        bound = 2.0 ** -8 * y.abs() + (1 + 2.0 ** -8) * ref.e4m3_sum_error(inp.x.shape[1]) * mag
        off = (got.double() - y).abs()[inp.real]
        assert (off <= bound[inp.real]).all(), (off / bound[inp.real]).max()
    assert (got[~inp.real] == ref.SENTINEL_OUT).all()
    assert (buf[:, n:] == ref.SENTINEL_OUT).all()
    return got


COUNTS = [
    [1],
    [0, 0, 1, 0],
    [0, 0, 0],
    [5, 0, 64, 65, 63, 1, 16, 17],
    [300, 1, 129, 0, 257],
    [15, 33, 0, 31, 32, 2, 47, 48, 49, 128, 127],
]


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("n,channels", [(32, 128), (128, 384), (160, 256), (1408, 896)])
def test_product_bit_exact_where_sums_are(moe, counts, n, channels):
    for align in (1, 128):
        inp = Inputs(counts, n, channels, align=align, extra=3, exact=True, seed=n + channels)
        if inp.cap:
            check_product(moe, inp, True)


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("n,channels", [(96, 128), (512, 1024)])
def test_product_general_values(moe, counts, n, channels):
    check_product(moe, Inputs(counts, n, channels, extra=1, seed=7), False)


def test_product_row_strides(moe):
    inp = Inputs([70, 3, 0, 130], 224, 256, exact=True, seed=3, pad=48)
    check_product(moe, inp, True, pad=24)


def test_product_longest_row_stride(moe):
    """Rows 2^23 bytes apart, in every tile's height (the sums are exact)."""
    inp = Inputs([260], 33280, 128, align=1, exact=True, seed=9)
    x, xs, w, ws, counts, send = inp.gpu
    far = torch.zeros((260, 1 << 23), dtype=torch.uint8, device=DEV)[:, :128]
    far.copy_(x)
    want = inp.product()[0].bfloat16()
    for n, r in ((33280, 260), (33280, 40), (96, 260), (4096, 260)):
        got = moe.moe_grouped_gemm_fp8(far, xs, w[:, :n].contiguous(),
                                       ws[:, :-(-n // 128)].contiguous(), counts, send,
                                       expected_rows=r, check=True)
        assert torch.equal(got.cpu(), want[:, :n])


@pytest.mark.parametrize("experts", [1, 2, 63, 256, 511, 512])
def test_product_many_experts(moe, experts):
    rng = np.random.default_rng(experts)
    counts = rng.integers(0, 6, experts)
    counts[rng.integers(0, experts)] = 150
    check_product(moe, Inputs(counts.tolist(), 64, 256, align=16, exact=True, seed=1), True)


def test_product_does_not_depend_on_expected_rows(moe):
    """Launch and tile shapes follow expected_rows; results do not."""
    inp = Inputs([200, 0, 3, 700, 16, 1], 288, 512, seed=5)
    got = [check_product(moe, inp, False, expected_rows=r)
           for r in (None, 0, 1, 40, 100, 300, 920, 5000, 10 ** 9)]
    for g in got[1:]:
        assert torch.equal(g.view(torch.int16), got[0].view(torch.int16))


@pytest.mark.parametrize("rows", [1, 20, 49])
def test_product_block_order(moe, rows):
    """4096 channels begin their sums at a block that follows the output
    channel; every tile shape adds up alike, also where a start wraps."""
    inp = Inputs([rows, 0, 3 * rows], 1440, 4096, align=1, exact=True, seed=rows)
    check_product(moe, inp, True)
    inp = Inputs([rows, 3], 1440, 4096, align=1, seed=rows)
    got = [check_product(moe, inp, False, expected_rows=r) for r in (2, 60, 400)]
    for g in got[1:]:
        assert torch.equal(g.view(torch.int16), got[0].view(torch.int16))


@pytest.mark.parametrize("per_expert", [16, 17, 48, 49])
def test_product_tile_rules(moe, per_expert):
    """Rows an expert on both sides of each change of tile, all of them full."""
    check_product(moe, Inputs([per_expert] * 5, 416, 384, exact=True, seed=per_expert), True,
                  expected_rows=5 * per_expert)


def test_product_every_tile(moe):
    """Each tile the rules know, on rows that fill, straddle and miss them."""
    rng = np.random.default_rng(61)
    counts = rng.integers(0, 70, 64)
    counts[[3, 9, 20]] = [0, 128, 1]
    inp = Inputs(counts.tolist(), 1056, 256, exact=True, seed=61)
    for r in (640, 1280, 3840, 8192):
        check_product(moe, inp, True, expected_rows=r)
    inp = Inputs(counts.tolist(), 1056, 384, seed=62)
    got = [check_product(moe, inp, False, expected_rows=r) for r in (640, 1280, 3840, 8192)]
    for g in got[1:]:
        assert torch.equal(g.view(torch.int16), got[0].view(torch.int16))
    few = Inputs([300, 0, 129, 640, 256], 1440, 384, align=1, seed=63)
    got = [check_product(moe, few, False, expected_rows=r) for r in (None, 500, 60)]
    for g in got[1:]:
        assert torch.equal(g.view(torch.int16), got[0].view(torch.int16))


@pytest.mark.parametrize("counts", [[1100], [600, 0, 1, 499], [1, 256, 257, 511, 75]])
def test_product_large_tiles(moe, counts):
    """Enough tiles that the largest shape is taken; the others agree with it."""
    check_product(moe, Inputs(counts, 7456, 256, align=16, exact=True, extra=5, seed=11), True,
                  expected_rows=1100)
    inp = Inputs(counts, 7456, 384, align=1, seed=12)
    got = [check_product(moe, inp, False, expected_rows=r) for r in (1100, 300, 1)]
    for g in got[1:]:
        assert torch.equal(g[inp.real].view(torch.int16), got[0][inp.real].view(torch.int16))


@pytest.mark.parametrize("rows", [1, 2, 17, 64, 300, 1111])
def test_dense_product(moe, rows):
    """Without counts: one group of every row."""
    inp = Inputs([rows], 352, 640, align=1, exact=True, seed=rows)
    x, xs, w, ws, _, _ = inp.gpu
    out = moe.moe_grouped_gemm_fp8(x, xs, w, ws, None, None)
    y, _ = inp.product()
    assert torch.equal(out.cpu(), y.bfloat16())
    empty = moe.moe_grouped_gemm_fp8(x[:0], xs[:0], w, ws, None, None)
    assert tuple(empty.shape) == (0, 352)


@pytest.mark.parametrize("n,channels", [(32, 65536), (65536, 128)])
def test_product_largest_features(moe, n, channels):
    check_product(moe, Inputs([3, 0, 18], n, channels, align=1, exact=True, seed=51), True,
                  expected_rows=21)


def test_product_non_finite_values_reach_their_own_outputs_only(moe):
    inp = Inputs([40, 40], 128, 256, exact=True, seed=9)
    clean = check_product(moe, inp, True)
    x, xs, w, ws, counts, send = inp.gpu
    x = x.clone()
    ws, xs = ws.clone(), xs.clone()
    x[3, 200] = 0x7F                    # NaN code in row 3
    xs[5, 1] = float("inf")
    ws[1, 0, 1] = float("nan")          # expert 1's one block of rows
    out = moe.moe_grouped_gemm_fp8(x, xs, w, ws, counts, send,
                                   out=torch.zeros((inp.cap, 128), dtype=torch.bfloat16,
                                                   device=DEV)).cpu()
    assert out[3].isnan().all()
    assert not out[5].isfinite().any()
    s1 = int(inp.send[1])
    assert out[s1:s1 + 40].isnan().all()
    keep = torch.ones(40, dtype=torch.bool)
    keep[3] = keep[5] = False
    assert torch.equal(out[:40][keep], clean[:40][keep])


def test_product_segments_beyond_the_buffer_are_guarded(moe):
    """Counts and offsets that leave the buffer: rows inside are computed, no
    row outside is touched, the status word says so."""
    inp = Inputs([50, 100], 64, 128, exact=True, seed=11)
    x, xs, w, ws, counts, send = inp.gpu
    y, _ = inp.product()
    cap = int(inp.send[1]) + 30          # the second segment is cut after 30 rows
    out = torch.full((inp.cap, 64), ref.SENTINEL_OUT, dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    moe.moe_grouped_gemm_fp8(x[:cap], xs[:cap], w, ws, counts, send, out=out[:cap], status=status)
    got = out.cpu()
    assert int(status.item()) == moe.MOE_FLAG_GUARD
    assert torch.equal(got[:50], y[:50].bfloat16())
    assert torch.equal(got[int(inp.send[1]):cap], y[int(inp.send[1]):cap].bfloat16())
    assert (got[cap:] == ref.SENTINEL_OUT).all()
    with pytest.raises(moe.MoeStatusError):
        moe.moe_grouped_gemm_fp8(x[:cap], xs[:cap], w, ws, counts, send, out=out[:cap],
                                 check=True)


@pytest.mark.parametrize("counts,send", [
    ([-5, 3], [0, 128, 256]),
    ([3, 3], [-4, 128, 256]),
    ([2 ** 31 - 1, 2 ** 31 - 1], [0, 0, 0]),
    ([1, 1], [2 ** 31 - 1, 255, 256]),
])
def test_product_bad_counts_stay_inside_the_buffer(moe, counts, send):
    inp = Inputs([128, 128], 64, 128, exact=True, seed=12)
    x, xs, w, ws, _, _ = inp.gpu
    out = torch.full((inp.cap + 8, 64), ref.SENTINEL_OUT, dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    moe.moe_grouped_gemm_fp8(x, xs, w, ws, torch.tensor(counts, dtype=torch.int32, device=DEV),
                             torch.tensor(send, dtype=torch.int32, device=DEV),
                             out=out[4:4 + inp.cap], status=status)
    assert int(status.item()) == moe.MOE_FLAG_GUARD
    got = out.cpu()
    assert (got[:4] == ref.SENTINEL_OUT).all() and (got[4 + inp.cap:] == ref.SENTINEL_OUT).all()


def test_product_overlapping_segments_write_nothing(moe):
    """More rows than the buffer holds: refused on the device."""
    e = 512
    x = torch.zeros((1024, 128), dtype=torch.uint8, device=DEV)
    xs = torch.ones((1024, 1), device=DEV)
    w = torch.zeros((e, 32, 128), dtype=torch.uint8, device=DEV)
    ws = torch.ones((e, 1, 1), device=DEV)
    out = torch.full((1024, 32), ref.SENTINEL_OUT, dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    moe.moe_grouped_gemm_fp8(x, xs, w, ws,
                             torch.full((e,), 1024, dtype=torch.int32, device=DEV),
                             torch.zeros(e + 1, dtype=torch.int32, device=DEV), out=out,
                             status=status)
    assert int(status.item()) == moe.MOE_FLAG_GUARD
    assert (out == ref.SENTINEL_OUT).all()


# ------------------------------------------------------------------ gated

def gated_reference(z, mag, channels):
    """h of a product z (with its terms' summed magnitudes) and a bound of its
    fp32 error, in float64."""
    inter = z.shape[1] // 2
    dz = ref.sum_error(channels) * mag
    g, u = z[:, :inter], z[:, inter:]
    dg, du = dz[:, :inter], dz[:, inter:]
    silu = g / (1 + torch.exp(-g))
    h = silu * u
    # |silu'| <= 1.1; the exponential's argument is rounded (2^-24 of |g| log2 e,
    # as a factor of the result), its value, the sum, the reciprocal and the two
    # products are each off by at most 2^-23.
    rel = (1.5 * g.abs() + 8) * 2.0 ** -23
    dh = (u.abs() + du) * 1.1 * dg + (silu.abs() + 1.1 * dg) * du + rel * h.abs()
    return h, dh


def check_gated(moe, inp, expected_rows=None, pad=0):
    inter = inp.w.shape[1] // 2
    buf = torch.full((inp.cap, inter + pad), ref.SENTINEL_CODE, dtype=torch.uint8, device=DEV)
    scales = torch.full((inp.cap, inter // 128), ref.SENTINEL_SCALE, device=DEV)
    codes, scales = moe.moe_grouped_gemm_silu_fp8(
        *inp.gpu, out=buf[:, :inter], out_scales=scales, expected_rows=expected_rows, check=True)
    codes, scales = codes.cpu(), scales.cpu()
    h, dh = gated_reference(*inp.product(), inp.x.shape[1])
    r = inp.real
    blocks = h.view(h.shape[0], -1, 128)
    want = blocks.abs().amax(2) / 448
    ds = dh.view(blocks.shape).amax(2) / 448 + 2.0 ** -23 * want
    off = (scales.double() - want).abs()
    assert (off <= ds)[r].all(), (off / ds)[r].max()
    # code * scale against h: half an e4m3 step, and what h and the scale are off by
    s = scales.double().repeat_interleave(128, 1)
    got = ref.values(codes) * s
    bound = 2.0 ** -4 * h.abs() + 2.0 ** -10 * s + 1.1 * dh \
        + 448 * ds.repeat_interleave(128, 1)
    off = (got - h).abs()
    assert (off <= bound)[r].all(), (off / bound)[r].max()
    assert (codes[~r] == ref.SENTINEL_CODE).all() and (scales[~r] == ref.SENTINEL_SCALE).all()
    assert (buf[:, inter:] == ref.SENTINEL_CODE).all()
    return codes, scales


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("inter,channels", [(128, 128), (384, 640)])
def test_gated_general_values(moe, counts, inter, channels):
    for align in (1, 128):
        inp = Inputs(counts, 2 * inter, channels, align=align, extra=2, seed=inter)
        if inp.cap:
            check_gated(moe, inp)


def test_gated_strides_and_expected_rows(moe):
    inp = Inputs([200, 0, 3, 70, 16, 1], 512, 512, seed=21, pad=32)
    got = [check_gated(moe, inp, r, pad=64) for r in (None, 1, 40, 100, 290, 10 ** 6)]
    for c, s in got[1:]:
        assert torch.equal(c, got[0][0]) and torch.equal(s, got[0][1])


@pytest.mark.parametrize("per_expert", [20, 21, 96, 97])
def test_gated_tile_rules(moe, per_expert):
    check_gated(moe, Inputs([per_expert] * 2, 512, 384, seed=per_expert),
                expected_rows=2 * per_expert)


def test_gated_every_tile(moe):
    rng = np.random.default_rng(64)
    counts = rng.integers(0, 128, 16)
    counts[[2, 5]] = [0, 128]
    inp = Inputs(counts.tolist(), 2048, 384, seed=64)
    got = [check_gated(moe, inp, r) for r in (160, 336, 960, 1600)]
    for c, s in got[1:]:
        assert torch.equal(c, got[0][0]) and torch.equal(s, got[0][1])


def test_gated_half_empty_tiles(moe):
    """Tiles of 64 rows whose second half, or all but one row, is missing."""
    rng = np.random.default_rng(65)
    counts = rng.integers(0, 80, 24)
    counts[[0, 1, 2, 3, 4, 5]] = [1, 32, 33, 64, 65, 97]
    inp = Inputs(counts.tolist(), 2048, 384, align=1, seed=65)
    got = [check_gated(moe, inp, r) for r in (960, 24, 24 * 60)]
    for c, s in got[1:]:
        assert torch.equal(c[inp.real], got[0][0][inp.real])
        assert torch.equal(s[inp.real], got[0][1][inp.real])


def test_gated_block_order(moe):
    inp = Inputs([3, 0, 60], 2048, 4096, align=1, seed=24)
    got = [check_gated(moe, inp, r) for r in (3, 63, 3 * 225)]
    for c, s in got[1:]:
        assert torch.equal(c[inp.real], got[0][0][inp.real])
        assert torch.equal(s[inp.real], got[0][1][inp.real])


@pytest.mark.parametrize("inter,channels", [(128, 65536), (32768, 128)])
def test_gated_largest_features(moe, inter, channels):
    check_gated(moe, Inputs([2, 17], 2 * inter, channels, align=1, seed=52), expected_rows=19)


def test_gated_dense(moe):
    inp = Inputs([77], 256, 384, align=1, seed=22)
    a = check_gated(moe, inp)
    codes, scales = moe.moe_grouped_gemm_silu_fp8(*inp.gpu[:4], None, None)
    assert torch.equal(codes.cpu(), a[0]) and torch.equal(scales.cpu(), a[1])


def test_gated_zero_and_non_finite_blocks(moe):
    """An all-zero row gives scale 0 and codes 0; a NaN or an infinity gives a
    non-finite scale and NaN codes in the blocks that hold it."""
    inp = Inputs([20], 512, 256, seed=23)
    x, xs, w, ws, counts, send = inp.gpu
    x, xs = x.clone(), xs.clone()
    x[4] = 0
    xs[6] = float("inf")
    x[8, 3] = 0x7F
    codes, scales = moe.moe_grouped_gemm_silu_fp8(x, xs, w, ws, counts, send)
    codes, scales = codes.cpu(), scales.cpu()
    assert (codes[4] == 0).all() and (scales[4] == 0).all()
    for row in (6, 8):
        assert not scales[row].isfinite().any()
        assert (codes[row] == 0x7F).all()
    ok = torch.ones(20, dtype=torch.bool)
    ok[[4, 6, 8]] = False
    clean = check_gated(moe, inp)
    assert torch.equal(codes[:20][ok], clean[0][:20][ok])


def test_gated_large_gates_saturate_like_the_formula(moe):
    """Gates far beyond the exponential's range: silu is 0 or the gate."""
    x = torch.full((2, 128), 0x38, dtype=torch.uint8)           # 1.0
    w = torch.full((1, 256, 128), 0x38, dtype=torch.uint8)
    xs = torch.tensor([[100.0], [-100.0]])                      # gates of +-12800
    ws = torch.ones((1, 2, 1))
    codes, scales = moe.moe_grouped_gemm_silu_fp8(x.to(DEV), xs.to(DEV), w.to(DEV), ws.to(DEV),
                                                  None, None)
    assert (ref.values(codes[0]) == 448).all()
    # 12800 * 12800 / 448: the product and the quotient each rounded once
    assert abs(float(scales[0, 0]) - 12800.0 ** 2 / 448) <= 12800.0 ** 2 / 448 * 2.0 ** -22
    assert (ref.values(codes[1]) == 0).all() and float(scales[1, 0]) == 0.0


# ------------------------------------------------------------------ the run of them

def quantised_weights(gen, e, n, channels):
    w = torch.randn((e, n, channels), generator=gen) / math.sqrt(channels)
    b = w.view(e, n // 128, 128, channels // 128, 128)
    s = b.abs().amax((2, 4)) / 448
    q = (b / s[:, :, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.view(e, n, channels), s


@pytest.mark.parametrize("bs,hidden,inter,e,k", [(1, 256, 128, 8, 2), (37, 384, 256, 12, 3),
                                                 (600, 256, 384, 16, 8)])
def test_served_layer(moe, bs, hidden, inter, e, k):
    """dispatch (e4m3) -> gated product -> product -> combine with a shared
    expert, as a serving loop runs it, captured once and replayed on new
    tokens; each stage against its 64-bit form on the stage's own inputs."""
    gen = torch.Generator().manual_seed(bs)
    w1, s1 = quantised_weights(gen, e, 2 * inter, hidden)
    w2, s2 = quantised_weights(gen, e, hidden, inter)
    d1, d2 = quantised_weights(gen, 1, 2 * inter, hidden)
    d3, d4 = quantised_weights(gen, 1, hidden, inter)
    on = [t.to(DEV) for t in (w1, s1, w2, s2, d1, d2, d3, d4)]
    x = torch.zeros((bs, hidden), dtype=torch.bfloat16, device=DEV)
    ids = torch.zeros((bs, k), dtype=torch.int32, device=DEV)
    scales = torch.zeros((bs, k), device=DEV)
    one = torch.zeros((bs, 1), dtype=torch.int32, device=DEV)
    ws = torch.zeros(max(moe.moe_dispatch_layout_workspace_size(bs, k, e), 16),
                     dtype=torch.uint8, device=DEV)
    ws1 = torch.zeros(max(moe.moe_dispatch_layout_workspace_size(bs, 1, 1), 16),
                      dtype=torch.uint8, device=DEV)

    def new_tokens(seed):
        g = torch.Generator().manual_seed(seed)
        x.copy_(torch.randn((bs, hidden), generator=g).bfloat16())
        ids.copy_(torch.rand((bs, e), generator=g).topk(k, 1).indices.int())
        scales.copy_(torch.softmax(torch.randn((bs, k), generator=g), 1))

    def layer():
        lay, ex, qs = moe.moe_dispatch_fused(x, ids, e, out_dtype="fp8", workspace=ws)
        h, hs = moe.moe_grouped_gemm_silu_fp8(ex, qs, on[0], on[1], lay.expert_counts,
                                              lay.ep_send_counts, expected_rows=bs * k)
        y = moe.moe_grouped_gemm_fp8(h, hs, on[2], on[3], lay.expert_counts,
                                     lay.ep_send_counts, expected_rows=bs * k)
        # the shared expert: every token to one expert, its rows dense
        _, sx, sq = moe.moe_dispatch_fused(x, one, 1, 1, out_dtype="fp8", workspace=ws1)
        sh, shs = moe.moe_grouped_gemm_silu_fp8(sx, sq, on[4], on[5], None, None)
        shared = moe.moe_grouped_gemm_fp8(sh, shs, on[6], on[7], None, None)
        out = moe.moe_combine(y, ids, lay.expand_idx, lay.ep_send_counts, scales, shared, e)
        return lay, ex, qs, h, hs, y, sx, sq, sh, shs, shared, out

    new_tokens(1)
    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = layer()
    for seed in (2, 3, 4):
        new_tokens(seed)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() if torch.is_tensor(t) else t for t in kept]
        eager = layer()
        torch.cuda.synchronize()
        lay, ex, qs, h, hs, y, sx, sq, sh, shs, shared, out = got
        counts = kept[0].expert_counts.cpu().tolist()
        send = kept[0].ep_send_counts.cpu().numpy()
        real = ref.real_rows(ex.shape[0], counts, send)
        for a, b in zip(got[1:6], eager[1:6]):
            assert torch.equal(a.cpu()[real], b.cpu()[real])
        assert torch.equal(out, eager[-1]) and torch.equal(shared, eager[-2])

        def stage(codes, qscales, w, s, c, o, real):
            v = ref.dequantised(codes, qscales)
            v[~real] = 0
            return ref.product(v, ref.weight_values(w, s), c, o)

        def near_product(got, y64, mag, channels, real):
            bound = 2.0 ** -8 * y64.abs() + (1 + 2.0 ** -8) * ref.e4m3_sum_error(channels) * mag
            assert ((got.cpu().double() - y64).abs() <= bound)[real].all()

        y64, mag = stage(h, hs, w2, s2, counts, send, real)
        near_product(y, y64, mag, inter, real)
        every = torch.ones(bs, dtype=torch.bool)
        y64, mag = stage(sh, shs, d3, d4, [bs], [0, bs], every)
        near_product(shared, y64, mag, inter, every)
        h64, dh = gated_reference(*stage(ex, qs, w1, s1, counts, send, real), hidden)
        # half an e4m3 step, what h is off by, and the scale's and its own roundings
        bound = (2.0 ** -4 + 2.0 ** -22) * h64.abs() + 1.1 * dh \
            + 2.0 ** -10 * hs.cpu().double().repeat_interleave(128, 1) \
            + dh.view(*dh.shape[:1], -1, 128).amax(2).repeat_interleave(128, 1)
        assert ((ref.dequantised(h, hs) - h64).abs() <= bound)[real].all()


@pytest.mark.parametrize("gated", [False, True])
def test_streams_and_prepared_calls(moe, gated):
    """Two streams with work in flight on both, and a prepared call repeated
    on new contents: each equals the call alone."""
    entry = moe.moe_grouped_gemm_silu_fp8 if gated else moe.moe_grouped_gemm_fp8
    a = Inputs([130, 5, 0, 260], 512, 512, seed=31)
    b = Inputs([3, 300, 77, 1], 512, 512, seed=32)

    def first(v):
        return v[0] if gated else v

    want = [first(entry(*i.gpu)).cpu() for i in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(4):
        for i, (inp, st) in enumerate(zip((a, b), streams)):
            with torch.cuda.stream(st):
                outs[i].append(first(entry(*inp.gpu)))
    torch.cuda.synchronize()
    for i, inp in enumerate((a, b)):
        for o in outs[i]:
            assert torch.equal(o.cpu()[inp.real].view(torch.uint8),
                               want[i][inp.real].view(torch.uint8))
    call = moe.prepare(entry, *a.gpu, expected_rows=395)
    for src in (b, a):
        if src is b:
            a.gpu[2].copy_(b.gpu[2])
        else:
            a.gpu[2].copy_(a.w)
        call()
        torch.cuda.synchronize()
    assert torch.equal(first(call.result).cpu()[a.real].view(torch.uint8),
                       want[0][a.real].view(torch.uint8))


def test_product_past_four_gigabytes(moe):
    """Weights, rows and outputs whose byte offsets pass 2^32: the last expert
    and the last rows equal the same product on a copy of that expert alone."""
    gen = torch.Generator().manual_seed(41)
    e, n, channels = 66, 8192, 8192                  # 4.4e9 bytes of weights
    w = torch.zeros((e, n, channels), dtype=torch.uint8, device=DEV)
    w[-1].copy_(ref.small_codes(gen, (n, channels)))
    ws = torch.ones((e, n // 128, channels // 128), device=DEV)
    rows = 530_000                                   # 4.3e9 bytes of rows, 8.7e9 of outputs
    x = torch.zeros((rows, channels), dtype=torch.uint8, device=DEV)
    x[-40:].copy_(ref.small_codes(gen, (40, channels)))
    xs = torch.ones((rows, channels // 128), device=DEV)
    counts = torch.zeros(e, dtype=torch.int32, device=DEV)
    counts[-1] = 37
    send = torch.zeros(e + 1, dtype=torch.int32, device=DEV)
    send[1:] = rows - 40
    out = torch.zeros((rows, n), dtype=torch.bfloat16, device=DEV)
    moe.moe_grouped_gemm_fp8(x, xs, w, ws, counts, send, out=out, expected_rows=37)
    y = ref.values(x[-40:-3]) @ ref.values(w[-1]).t()
    assert torch.equal(out[-40:-3].cpu(), y.bfloat16())
    assert (out[-3:] == 0).all() and (out[-100:-40] == 0).all()
