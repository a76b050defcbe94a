"""Refusals of the experts' products and of the path's gradient, on the CPU:
the Python binding's checks with the library stubbed (a refused call never
reaches it), and the C ABI's own rules (a refused call enqueues nothing, so
none of these needs a GPU)."""

import ctypes

import pytest
import torch

import combine_moe_dispatch_layout_amd as moe
from test_binding_checks import StubLib, bf16, expect_refused, f32, i32

BS, K, E, H, CAP = 40, 4, 8, 256, 512
N, C = 288, 384


@pytest.fixture
def stub(monkeypatch):
    lib = StubLib()
    monkeypatch.setattr(moe, "_DEVICE_TYPE", "cpu")
    monkeypatch.setattr(moe, "load_library", lambda: lib)
    monkeypatch.setattr(moe, "_stream", lambda t: None)
    return lib


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def product(entry="moe_grouped_gemm_fp8", **kw):
    n = kw.pop("n", N if entry == "moe_grouped_gemm_fp8" else 512)
    args = dict(expand_x=u8(CAP, C), quant_scales=f32(CAP, C // 128), weight=u8(E, n, C),
                weight_scales=f32(E, -(-n // 128), C // 128), expert_counts=i32(E),
                ep_send_counts=i32(E + 1))
    args.update(kw)
    return lambda: getattr(moe, entry)(**args)


@pytest.mark.parametrize("entry", ["moe_grouped_gemm_fp8", "moe_grouped_gemm_silu_fp8"])
def test_product_good_calls(stub, entry):
    product(entry)()
    product(entry, expand_x=u8(CAP, C + 64)[:, :C], expected_rows=160)()
    product(entry, weight=u8(1, 512, C), weight_scales=f32(1, 4, 3), expert_counts=None,
            ep_send_counts=None)()
    assert stub.calls == [entry] * 3


COMMON = [
    (dict(expand_x=bf16(CAP, C)), "expand_x must be"),
    (dict(expand_x=u8(CAP, C).t()), "unit column stride"),
    (dict(expand_x=u8(CAP, C + 1)), "multiple of 128"),
    (dict(expand_x=u8(CAP, 0)), "multiple of 128"),
    (dict(quant_scales=f32(CAP, C // 128 + 1)), "quant_scales must be"),
    (dict(quant_scales=f32(CAP - 1, C // 128)), "quant_scales must be"),
    (dict(quant_scales=f32(C // 128, CAP).t()), "contiguous"),
    (dict(weight=u8(E, 512, C + 128)), "weight must be"),
    (dict(weight=u8(512, C)), "weight must be"),
    (dict(weight=torch.zeros((E, 512, C), dtype=torch.int8)), "weight must be"),
    (dict(weight_scales=f32(E, 5, C // 128)), "weight_scales must be"),
    (dict(weight_scales=f32(E - 1, 4, C // 128)), "weight_scales must be"),
    (dict(expert_counts=None), "go together"),
    (dict(ep_send_counts=None), "go together"),
    (dict(expert_counts=None, ep_send_counts=None), "one expert"),
    (dict(expert_counts=i32(E - 1)), "expert_counts holds"),
    (dict(ep_send_counts=i32(E)), "ep_send_counts holds"),
    (dict(expert_counts=torch.zeros(E, dtype=torch.int64)), "expert_counts must be"),
    (dict(expected_rows=-1), "expected_rows"),
    (dict(status=f32(1)), "status must be"),
]


@pytest.mark.parametrize("entry", ["moe_grouped_gemm_fp8", "moe_grouped_gemm_silu_fp8"])
@pytest.mark.parametrize("kw,match", COMMON)
def test_product_refusals(stub, entry, kw, match):
    expect_refused(stub, product(entry, n=512, **kw), match)


@pytest.mark.parametrize("entry,kw,match", [
    ("moe_grouped_gemm_fp8", dict(out=f32(CAP, N)), "out must be"),
    ("moe_grouped_gemm_fp8", dict(out=bf16(CAP - 1, N)), "out has"),
    ("moe_grouped_gemm_fp8", dict(out=bf16(CAP, N + 8)), "columns"),
    ("moe_grouped_gemm_silu_fp8", dict(n=384), "multiple of 128"),
    ("moe_grouped_gemm_silu_fp8", dict(n=0), "multiple of 128"),
    ("moe_grouped_gemm_silu_fp8", dict(out=bf16(CAP, 256)), "out must be"),
    ("moe_grouped_gemm_silu_fp8", dict(out=u8(CAP, 512)), "columns"),
    ("moe_grouped_gemm_silu_fp8", dict(out_scales=f32(CAP, 3)), "columns"),
    ("moe_grouped_gemm_silu_fp8", dict(out_scales=f32(CAP - 1, 2)), "out_scales has"),
])
def test_product_output_refusals(stub, entry, kw, match):
    expect_refused(stub, product(entry, **kw), match)


def backward(**kw):
    args = dict(grad_out=bf16(BS, H), expand_x=bf16(CAP, H), expert_ids=i32(BS, K),
                expand_idx=i32(BS * K), ep_send_counts=i32(E + 1), expert_scales=f32(BS, K),
                num_experts=E)
    args.update(kw)
    return lambda: moe.moe_combine_backward(**args)


def test_backward_good_calls(stub):
    dy, dw = backward()()
    assert tuple(dy.shape) == (CAP, H) and tuple(dw.shape) == (BS, K)
    assert backward(need_expand_x=False)()[0] is None
    assert backward(need_scales=False, expand_x=None, capacity_rows=CAP)()[1] is None
    backward(need_scales=False, expand_x=None, grad_expand_x=bf16(CAP, H))()
    moe.moe_dispatch_backward(bf16(CAP, H), i32(BS, K), i32(BS * K), i32(E + 1), E,
                              grad_x_add=bf16(BS, H))
    assert stub.calls == ["moe_combine_backward"] * 4 + ["moe_dispatch_backward"]


@pytest.mark.parametrize("kw,match", [
    (dict(grad_out=f32(BS, H)), "grad_out must be"),
    (dict(grad_out=bf16(BS * H)), r"\[BS, H\]"),
    (dict(expand_x=None), "expand_x is needed"),
    (dict(expand_x=None, need_scales=False), "must give the rows"),
    (dict(expand_x=bf16(CAP, H + 8)), "columns"),
    (dict(expand_x=bf16(CAP, H), capacity_rows=CAP + 1), "expand_x has"),
    (dict(capacity_rows=-1), "capacity_rows"),
    (dict(expert_ids=i32(BS + 1, K)), "rows, x has"),
    (dict(expand_idx=i32(BS * K - 1)), "expand_idx holds"),
    (dict(ep_send_counts=i32(E)), "ep_send_counts holds"),
    (dict(expert_scales=f32(BS * K - 1)), "expert_scales holds"),
    (dict(need_expand_x=False, need_scales=False), "must be set"),
    (dict(grad_expand_x=bf16(CAP - 1, H)), "grad_expand_x has"),
    (dict(grad_expand_x=f32(CAP, H)), "grad_expand_x must be"),
    (dict(grad_expert_scales=f32(BS, K + 1)), "grad_expert_scales must be"),
    (dict(grad_expert_scales=bf16(BS, K)), "grad_expert_scales must be"),
])
def test_combine_backward_refusals(stub, kw, match):
    expect_refused(stub, backward(**kw), match)


@pytest.mark.parametrize("kw,match", [
    (dict(grad_expand_x=f32(CAP, H)), "grad_expand_x must be"),
    (dict(grad_expand_x=bf16(CAP * H)), "2-D"),
    (dict(expert_ids=i32(BS * K)), r"\[BS, K\]"),
    (dict(grad_x_add=bf16(BS - 1, H)), "grad_x_add has"),
    (dict(grad_x_add=bf16(BS, H + 8)), "columns"),
    (dict(out=bf16(BS, H + 8)), "out must be"),
    (dict(out=f32(BS, H)), "out must be"),
])
def test_dispatch_backward_refusals(stub, kw, match):
    args = dict(grad_expand_x=bf16(CAP, H), expert_ids=i32(BS, K), expand_idx=i32(BS * K),
                ep_send_counts=i32(E + 1), num_experts=E)
    args.update(kw)
    expect_refused(stub, lambda: moe.moe_dispatch_backward(**args), match)


# ------------------------------------------------------------------ the C ABI's rules

FAKE = 0x100000  # a non-null, 16-byte aligned address that no refused call touches
FAKE_OUT = 0x200000


@pytest.fixture(scope="module")
def lib():
    return moe.load_library()


PRODUCT = dict(x=FAKE, xs=C, cap=CAP, qs=FAKE, w=FAKE, ws=FAKE, counts=FAKE, send=FAKE, e=E, k=C,
               n=256, rows=0, out=FAKE_OUT, os=256, scales=FAKE, status=None, stream=None)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kw", [
    dict(e=0), dict(e=513), dict(k=0), dict(k=100), dict(k=-128), dict(k=65664, xs=65664),
    dict(n=0), dict(n=-128), dict(n=131072, os=131072), dict(n=144 - 8, os=144),
    dict(cap=-1), dict(cap=(1 << 30) + 1), dict(cap=1 << 30, n=1152, os=1152),
    dict(xs=(1 << 23) + 16), dict(rows=-1), dict(counts=None), dict(send=None),
    dict(counts=None, send=None), dict(x=None), dict(x=FAKE + 8), dict(xs=C - 16), dict(xs=C + 8),
    dict(w=None), dict(w=FAKE + 4), dict(qs=None), dict(qs=FAKE + 2), dict(ws=None),
    dict(out=None), dict(out=FAKE_OUT + 2), dict(out=FAKE), dict(os=248), dict(os=260),
])
def test_product_rules(lib, gated, kw):
    a = dict(PRODUCT)
    a.update(kw)
    args = [a[v] for v in ("x", "xs", "cap", "qs", "w", "ws", "counts", "send", "e", "k", "n",
                           "rows", "out", "os")]
    if gated:
        assert lib.moe_grouped_gemm_silu_fp8(*args, a["scales"], a["status"], a["stream"]) == 1
    else:
        assert lib.moe_grouped_gemm_fp8(*args, a["status"], a["stream"]) == 1


def test_product_rules_of_one_form(lib):
    a = dict(PRODUCT)
    names = ("x", "xs", "cap", "qs", "w", "ws", "counts", "send", "e", "k", "n", "rows", "out",
             "os")
    assert lib.moe_grouped_gemm_silu_fp8(*[a[v] for v in names], None, None, None) == 1
    a["n"] = 160   # a product may have it, the gated form not
    assert lib.moe_grouped_gemm_silu_fp8(*[a[v] for v in names], FAKE, None, None) == 1
    a["cap"] = 0   # no rows: nothing to do, whatever the pointers
    a.update(n=256, x=None, out=None)
    assert lib.moe_grouped_gemm_fp8(*[a[v] for v in names], None, None) == 0


BACK = dict(g=FAKE, gs=H, y=FAKE, ys=H, cap=CAP, ids=FAKE, idx=FAKE, send=FAKE, w=FAKE, bs=BS, h=H,
            k=K, e=E, dy=FAKE, dys=H, dw=FAKE, status=None, stream=None)


@pytest.mark.parametrize("kw", [
    dict(bs=-1), dict(k=0), dict(k=17, e=64), dict(k=9), dict(e=0), dict(e=513), dict(h=0),
    dict(h=48), dict(h=65568), dict(cap=-1), dict(ids=None), dict(idx=None), dict(send=None),
    dict(w=None), dict(g=None), dict(g=FAKE + 8), dict(gs=H - 8), dict(gs=H + 4), dict(y=None),
    dict(ys=H + 4), dict(dys=H - 32), dict(dw=FAKE + 2), dict(dy=None, dw=None),
    dict(bs=1 << 26, h=65536),
])
def test_combine_backward_rules(lib, kw):
    a = dict(BACK)
    a.update(kw)
    assert lib.moe_combine_backward(*a.values()) == 1


@pytest.mark.parametrize("kw", [
    dict(bs=-1), dict(k=0), dict(e=0), dict(h=48), dict(cap=-1), dict(ids=None), dict(idx=None),
    dict(send=None), dict(g=None), dict(gs=H + 4), dict(add=FAKE + 8), dict(adds=H - 8),
    dict(out=None), dict(out=FAKE + 8), dict(out=FAKE + 4096, add=FAKE + 4096),
])
def test_dispatch_backward_rules(lib, kw):
    a = dict(g=FAKE, gs=H, cap=CAP, ids=FAKE, idx=FAKE, send=FAKE, add=FAKE + 65536, adds=H, bs=BS,
             h=H, k=K, e=E, out=FAKE, status=None, stream=None)
    a.update(kw)
    assert lib.moe_dispatch_backward(*a.values()) == 1


def test_empty_batches_are_accepted_without_buffers(lib):
    a = dict(BACK)
    a.update(bs=0, g=None, y=None, ids=None, idx=None, send=None, w=None, dy=None, dw=None)
    assert lib.moe_combine_backward(*a.values()) == 0
    assert lib.moe_dispatch_backward(None, H, 0, None, None, None, None, 0, 0, H, K, E, None, None,
                                     None) == 0


def test_an_entry_on_another_device_makes_it_current(monkeypatch):
    """A call on tensors of a device that is not current switches to it for
    the launch, and back."""
    seen = []
    current = [0]

    class Guard:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            self.was, current[0] = current[0], self.dev

        def __exit__(self, *exc):
            current[0] = self.was

    monkeypatch.setattr(moe, "_get_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", Guard)

    def fn(*args):
        seen.append((current[0], args))
        return 0

    fn.argtypes = [ctypes.c_int]
    on1 = moe._on_device(fn, 1)
    assert on1.argtypes == fn.argtypes
    assert on1(5) == 0 and moe._on_device(fn, 0)(6) == 0
    assert seen == [(1, (5,)), (0, (6,))] and current[0] == 0
