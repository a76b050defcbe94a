"""Buffers of the path's gradient that share memory: refused, but for the two
in-place forms; and its other rules on buffers of their own, so that each
refusal has the one cause it names.  On the CPU: no call reaches a GPU."""

import pytest
import torch

import combine_moe_dispatch_layout_amd as moe

BS, K, E, H, CAP = 40, 4, 8, 256, 512
ROW = 2 * H
MB = 1 << 20
G, Y, IDS, IDX, SEND, W, DY, DW = (MB * i for i in range(1, 9))

# No call of these tests may reach a GPU: the addresses are made up.
no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="would launch on made-up rows")


@pytest.fixture(scope="module")
def lib():
    return moe.load_library()


def combine_backward(lib, **kw):
    a = dict(g=G, gs=H, y=Y, ys=H, cap=CAP, ids=IDS, idx=IDX, send=SEND, w=W, bs=BS, h=H, k=K, e=E,
             dy=DY, dys=H, dw=DW, status=None, stream=None)
    a.update(kw)
    return lib.moe_combine_backward(*a.values())


def dispatch_backward(lib, **kw):
    a = dict(g=Y, gs=H, cap=CAP, ids=IDS, idx=IDX, send=SEND, add=G, adds=H, bs=BS, h=H, k=K, e=E,
             out=DY, status=None, stream=None)
    a.update(kw)
    return lib.moe_dispatch_backward(*a.values())


@no_gpu
@pytest.mark.parametrize("kw", [
    dict(),
    dict(dy=Y), dict(dw=W),                                  # in place
    dict(dy=None), dict(dw=None), dict(dw=None, y=None, ys=0),
    dict(dy=Y + ROW, ys=2 * H, dys=2 * H),                   # columns side by side
    dict(dy=G + ROW, gs=2 * H, dys=2 * H),
    dict(dy=G + BS * ROW), dict(dw=G + BS * ROW),            # right behind
    dict(dw=None, dy=Y, dys=H + 8),                          # y is not read then
    dict(dy=None, dw=W + 4),                                 # nor are the weights
])
def test_combine_backward_on_separate_buffers_passes_the_rules(lib, kw):
    """Status 4: the launch was tried, and failed for want of a GPU."""
    assert combine_backward(lib, **kw) == 4


@pytest.mark.parametrize("kw", [
    dict(dy=Y, dys=H + 8), dict(dy=Y + ROW), dict(dy=Y + 16), dict(dy=Y + CAP * ROW - 16),
    dict(dy=Y, ys=2 * H),
    dict(dy=G), dict(dy=G + (BS - 1) * ROW), dict(g=DY + 16 * ROW),
    dict(dy=IDS), dict(dy=IDX), dict(dy=SEND), dict(dy=W), dict(dy=DW), dict(dw=DY + ROW),
    dict(dw=G), dict(dw=Y + 4), dict(dw=IDS), dict(dw=IDX + 4 * (BS * K - 1)), dict(dw=SEND),
    dict(dw=W + 4), dict(dw=W - 4 * (BS * K - 1)),
])
def test_combine_backward_refuses_shared_memory(lib, kw):
    assert combine_backward(lib, **kw) == 1


@pytest.mark.parametrize("kw", [
    dict(bs=-1), dict(k=0), dict(k=17, e=64), dict(k=9), dict(e=0), dict(e=513), dict(h=0),
    dict(h=48), dict(h=65568), dict(cap=-1), dict(ids=None), dict(idx=None), dict(send=None),
    dict(w=None), dict(w=W + 2), dict(g=None), dict(g=G + 8), dict(gs=H - 8), dict(gs=H + 4),
    dict(y=None), dict(y=Y + 4), dict(ys=H + 4), dict(dy=DY + 8), dict(dys=H - 32), dict(dw=DW + 2),
    dict(dy=None, dw=None), dict(bs=1 << 26, h=65536),
])
def test_combine_backward_rules_one_by_one(lib, kw):
    assert combine_backward(lib, **kw) == 1


@no_gpu
@pytest.mark.parametrize("kw", [
    dict(), dict(add=None), dict(cap=0, g=None, gs=0), dict(out=Y + CAP * ROW),
    dict(out=G + BS * ROW),
])
def test_dispatch_backward_on_separate_buffers_passes_the_rules(lib, kw):
    assert dispatch_backward(lib, **kw) == 4


@pytest.mark.parametrize("kw", [
    dict(out=Y), dict(out=Y + (CAP - 1) * ROW), dict(out=Y - (BS - 1) * ROW), dict(out=G),
    dict(out=G + 16), dict(out=G + ROW, adds=2 * H), dict(out=IDS), dict(out=IDX), dict(out=SEND),
    dict(ids=DY + 4), dict(idx=DY + ROW), dict(send=DY + BS * ROW - 4),
])
def test_dispatch_backward_refuses_shared_memory(lib, kw):
    assert dispatch_backward(lib, **kw) == 1


@pytest.mark.parametrize("kw", [
    dict(bs=-1), dict(k=0), dict(e=0), dict(h=48), dict(cap=-1), dict(ids=None), dict(idx=None),
    dict(send=None), dict(g=None), dict(gs=H + 4), dict(add=G + 8), dict(adds=H - 8),
    dict(out=None), dict(out=DY + 8),
])
def test_dispatch_backward_rules_one_by_one(lib, kw):
    assert dispatch_backward(lib, **kw) == 1
