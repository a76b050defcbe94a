"""The norm's weight gradient where every sum is exact: each row counts, once.

Rows hold +1 and -1 and eps is 3, so the mean of squares is 1 and r = 1 / sqrt(4)
without a rounding; with whole numbers grad_out[t] * x[t] * r are halves whose
sum over the rows stays below 2^23: bit for bit, in any order."""

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def moe():
    import combine_moe_dispatch_layout_amd as m
    m.load_library()
    assert torch.cuda.is_available()
    return m


# Every spread of a row over threads, one workgroup and as many as leave a row of
# sums, one turn of them and many.
@pytest.mark.parametrize("bs,h", [(1, 32), (64, 128), (65, 128), (200003, 32), (40000, 128),
                                  (33, 256), (20011, 256), (9000, 512), (16, 1024), (17, 1024),
                                  (8197, 1024), (9, 2048), (4099, 2048), (2, 2080), (3, 2080),
                                  (2501, 2080), (1029, 4096), (513, 4128), (2, 7168),
                                  (3, 7168), (1100, 7168), (530, 16416), (300, 32800),
                                  (259, 65536)])
def test_each_row_counts_once(moe, bs, h):
    gen = torch.Generator().manual_seed(bs + h)
    z = 2 * torch.randint(0, 2, (bs, h), generator=gen, dtype=torch.int8) - 1
    dy = torch.randint(-16, 17, (bs, h), generator=gen, dtype=torch.int8)
    dy[-3:] = torch.arange(h).remainder(97).add(11).to(torch.int8)   # the last rows stand out
    w = torch.ones(h, dtype=torch.bfloat16, device=DEV)
    zd, dyd = z.to(DEV).bfloat16(), dy.to(DEV).bfloat16()
    want = (z * dy).sum(0, dtype=torch.int64).double() / 2
    for need_x in (True, False):
        _, dw = moe.moe_rms_norm_backward(dyd, zd, w, eps=3.0, need_x=need_x)
        assert torch.equal(dw.cpu().double(), want)


def test_no_rows_and_no_pointers(moe):
    """With no rows nothing is read: the C ABI takes NULL for all that would be,
    and the weight's gradient becomes 0."""
    lib, stream = moe.load_library(), torch.cuda.current_stream().cuda_stream
    for h in (32, 256, 2048, 7168, 65536):
        for dtype in (moe.MOE_BF16, moe.MOE_FP32):
            dw = torch.full((h,), 5.0, device=DEV)
            assert lib.moe_rms_norm_backward(None, 0, None, 0, None, dtype, 0, h, 1e-6, None, 0,
                                             None, 0, dw.data_ptr(), None, 0,
                                             stream) == moe.MOE_OK
            assert (dw == 0).all()
    dw = torch.full((8, 64), 5.0, device=DEV)
    assert lib.moe_router_logits_backward(None, 0, None, 0, None, None, 0, 0, 64, 8, None, 0,
                                          dw.data_ptr(), None, 0, stream) == moe.MOE_OK
    assert (dw == 0).all()
