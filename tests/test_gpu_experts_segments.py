"""The experts' products on segments that share rows, on the GPU: two experts
with a row in common are refused on the device (flagged, nothing written), by
one row as by many and whatever tile expected_rows chooses; disjoint segments
in any order are computed.  The sums are exact, so results are compared bit
for bit."""

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


class Call:
    def __init__(self, moe, counts, send, cap, n, gated, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.moe, self.gated, self.cap = moe, gated, cap
        e = len(counts)
        self.counts, self.send = counts, send
        self.x = ref.small_codes(gen, (cap, 128))
        self.xs = ref.power_scales(gen, (cap, 1))
        self.w = ref.small_codes(gen, (e, n, 128))
        self.ws = ref.power_scales(gen, (e, -(-n // 128), 1))
        self.args = [t.to(DEV) for t in (self.x, self.xs, self.w, self.ws)]
        self.args += [torch.tensor(counts, dtype=torch.int32, device=DEV),
                      torch.tensor(send, dtype=torch.int32, device=DEV)]

    def __call__(self, expected_rows=None):
        """The outputs, as bytes, and the status word."""
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        n = self.w.shape[1]
        if self.gated:
            out = torch.full((self.cap, n // 2), ref.SENTINEL_CODE, dtype=torch.uint8, device=DEV)
            scales = torch.full((self.cap, n // 256), ref.SENTINEL_SCALE, device=DEV)
            self.moe.moe_grouped_gemm_silu_fp8(*self.args, out=out, out_scales=scales,
                                               status=status, expected_rows=expected_rows)
            return [out.cpu(), scales.cpu()], int(status.item())
        out = torch.full((self.cap, n), ref.SENTINEL_OUT, dtype=torch.bfloat16, device=DEV)
        self.moe.moe_grouped_gemm_fp8(*self.args, out=out, status=status,
                                      expected_rows=expected_rows)
        return [out.cpu()], int(status.item())

    def untouched(self, outs):
        if self.gated:
            return (outs[0] == ref.SENTINEL_CODE).all() and (outs[1] == ref.SENTINEL_SCALE).all()
        return (outs[0] == ref.SENTINEL_OUT).all()


ROWS = (None, 1, 40, 130, 600, 1100)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("counts,send,cap", [
    ([96, 96], [0, 0, 128], 128),               # more rows than the buffer, few tiles
    ([65, 64], [0, 64, 128], 128),              # one row in common
    ([128, 128], [0, 0, 256], 256),             # the same segment twice, within the buffer
    ([1, 1], [7, 7, 8], 128),                   # one row each
    ([600, 500, 1], [0, 600, 599], 1200),       # not the neighbour's, and out of order
    ([600, 0, 600], [500, 0, 0], 1200),         # a later one in front, reaching into it
    ([40, 0, 2 ** 31 - 1], [1190, 0, 1100], 1200),   # beyond the buffer's end as well
])
def test_segments_with_a_row_in_common_write_nothing(moe, gated, counts, send, cap):
    call = Call(moe, counts, send + [cap] * (len(counts) + 1 - len(send)), cap, 2048, gated)
    for rows in ROWS:
        outs, flags = call(rows)
        assert flags == moe.MOE_FLAG_GUARD, rows
        assert call.untouched(outs), rows


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("pair", [(0, 511), (3, 64), (63, 64), (254, 255), (255, 256), (130, 131)])
def test_two_of_many_segments_with_a_row_in_common(moe, gated, pair):
    """Experts held by one thread, by neighbouring ones and by other waves."""
    counts = [2] * 512
    send = [3 * e for e in range(513)]
    first = Call(moe, counts, send, 1600, 256, gated)
    want, flags = first()
    assert flags == 0
    send = list(send)
    send[pair[1]] = send[pair[0]] + 1
    call = Call(moe, counts, send, 1600, 256, gated)
    for rows in (None, 512, 40000):
        outs, flags = call(rows)
        assert flags == moe.MOE_FLAG_GUARD and call.untouched(outs)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("counts,send,cap", [
    ([300, 0, 129, 64], [129, 200, 0, 429, 500], 500),   # disjoint, in another order
    ([64, 0, 64, 0], [0, 32, 64, 64, 128], 128),         # empty ones inside others
    ([0, 128, 0], [5, 0, 128, 128], 128),
])
def test_disjoint_segments_are_computed_in_any_order(moe, gated, counts, send, cap):
    call = Call(moe, counts, send, cap, 768, gated, seed=5)
    x = ref.dequantised(call.x, call.xs)
    y, _ = ref.product(x, ref.weight_values(call.w, call.ws), counts, send)
    real = ref.real_rows(cap, counts, send)
    first = None
    for rows in ROWS:
        outs, flags = call(rows)
        assert flags == 0
        if not gated:
            assert torch.equal(outs[0][real], y[real].bfloat16())
            assert (outs[0][~real] == ref.SENTINEL_OUT).all()
        else:
            assert (outs[0][~real] == ref.SENTINEL_CODE).all()
            assert (outs[1][~real] == ref.SENTINEL_SCALE).all()
            want = torch.nn.functional.silu(y[:, :384]) * y[:, 384:]
            want = want.view(cap, 3, 128).abs().amax(2) / 448
            # the sums are exact and a block's largest has a gate over -87: the rounding
            # of the exponential's argument is a factor of 1.5 * 87 * 2^-23 at most, and
            # eight other operations are off by 2^-23 each, the quotient by 448 by 2^-24
            assert ((outs[1].double() - want).abs() <= 140 * 2.0 ** -23 * want)[real].all()
        first = outs if first is None else first
        assert all(torch.equal(a, b) for a, b in zip(outs, first))


def test_check_raises_on_a_row_in_common(moe):
    call = Call(moe, [65, 64], [0, 64, 128], 128, 256, False)
    with pytest.raises(moe.MoeStatusError):
        moe.moe_grouped_gemm_fp8(*call.args, check=True)
