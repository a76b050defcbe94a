"""Outputs of the experts' products that share memory with an input or with
each other are refused, through the C ABI and through the binding; columns of
one wider buffer side by side are not.  On the CPU: no call reaches a GPU."""

import ctypes

import pytest
import torch

import combine_moe_dispatch_layout_amd as moe

E, CAP, K, N = 3, 512, 256, 512
MB = 1 << 20
# Addresses 1 MB apart, larger than any buffer here.
X, QS, W, WS, COUNTS, SEND, OUT, SCALES = (MB * i for i in range(1, 9))


@pytest.fixture(scope="module")
def lib():
    return moe.load_library()


def call(lib, gated, **kw):
    a = dict(x=X, xs=K, cap=CAP, qs=QS, w=W, ws=WS, counts=COUNTS, send=SEND, e=E, k=K, n=N, rows=0,
             out=OUT, os=N)
    scales = kw.pop("scales", SCALES)
    a.update(kw)
    if gated:
        return lib.moe_grouped_gemm_silu_fp8(*a.values(), scales, None, None)
    return lib.moe_grouped_gemm_fp8(*a.values(), None, None)


# No call of these tests may reach a GPU: the addresses are made up.
no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="would launch on made-up rows")


@no_gpu
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kw", [
    dict(),
    dict(out=X + K, xs=2 * K + 1024, os=K + 512),                 # plain: beside x's columns
    dict(x=OUT + 2 * N, xs=2 * N + K, os=N + K // 2),             # and before them
    dict(out=X + CAP * K),                                        # right behind x
    dict(x=OUT - CAP * K),
])
def test_separate_buffers_pass_the_rules(lib, gated, kw):
    """Status 4: the launch was tried, and failed for want of a GPU."""
    if gated and "os" in kw:
        kw = dict(kw, os=kw["xs"])
        if "x" in kw:
            kw["x"] = OUT + N
    assert call(lib, gated, **kw) == 4


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kw", [
    dict(out=X), dict(out=X + 16), dict(out=X + CAP * K - 16), dict(x=OUT + 16 * N),
    dict(out=X + K - 16, xs=2 * K + 1024, os=K + 512),            # columns that meet
    dict(x=OUT + 2 * N - 16, xs=2 * N + K, os=N + K // 2),
    dict(out=QS), dict(out=QS + CAP * K // 128 * 4 - 16), dict(qs=OUT + 4),
    dict(out=W), dict(out=W + E * N * K - 16), dict(out=WS), dict(out=COUNTS), dict(out=SEND),
    dict(ws=OUT + 256), dict(counts=OUT + 4 * 100), dict(send=OUT + 4 * 100),
])
def test_out_over_an_input_is_refused(lib, gated, kw):
    if gated and "os" in kw:
        kw = dict(kw, os=kw["xs"])
        if "x" in kw:
            kw["x"] = OUT + N - 16
    assert call(lib, gated, **kw) == 1


@pytest.mark.parametrize("kw", [
    dict(scales=QS), dict(scales=QS + CAP * K // 128 * 4 - 4), dict(scales=X), dict(scales=W + 8),
    dict(scales=WS), dict(scales=COUNTS), dict(scales=SEND), dict(scales=OUT),
    dict(scales=OUT + CAP * N - 4), dict(out=SCALES + 16), dict(qs=SCALES - 4),
])
def test_out_scales_over_an_input_or_the_codes_are_refused(lib, kw):
    assert call(lib, True, **kw) == 1


def test_the_binding_raises(monkeypatch):
    """inter = hidden, so the rows' scales have the outputs' shape."""
    monkeypatch.setattr(moe, "_DEVICE_TYPE", "cpu")
    monkeypatch.setattr(moe, "_stream", lambda t: None)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    qs = torch.ones((CAP, K // 128))
    args = (u8(CAP, K), qs, u8(E, 2 * K, K), torch.ones((E, 2 * K // 128, K // 128)),
            torch.zeros(E, dtype=torch.int32), torch.zeros(E + 1, dtype=torch.int32))
    with pytest.raises(moe.MoeError) as e:
        moe.moe_grouped_gemm_silu_fp8(*args, out_scales=qs)
    assert e.value.code == moe.MOE_ERR_INVALID_ARG
    with pytest.raises(moe.MoeError) as e:
        moe.moe_grouped_gemm_silu_fp8(*args, out=args[0])
    assert e.value.code == moe.MOE_ERR_INVALID_ARG
