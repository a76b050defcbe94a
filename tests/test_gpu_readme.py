"""README's served layer and its gradient run as they are written."""

import os
import re

import pytest
import torch

import router_reference as ref
from router_reference import UBF16

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = "cuda"


def block(after):
    """The first Python block behind a line of README.md."""
    with open(os.path.join(ROOT, "README.md")) as f:
        text = f.read()
    return re.search(r"```python\n(.*?)```", text[text.index(after):], re.S).group(1)


def test_served_layer_and_gradient():
    import combine_moe_dispatch_layout_amd as moe
    gen = torch.Generator().manual_seed(0)
    bs, hidden, inter, experts, k = 24, 256, 128, 32, 8

    def normal(*shape):
        return torch.randn(shape, generator=gen)

    def codes(*shape):
        return normal(*shape).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)

    residual, a = normal(bs, hidden).bfloat16(), normal(bs, hidden).bfloat16()
    grad_residual = normal(bs, hidden).bfloat16()
    w = (1 + 0.1 * normal(hidden)).bfloat16()
    rows = moe.moe_dispatch_capacity(bs, k, experts, 128)
    names = dict(
        moe=moe, num_experts=experts, h=residual.to(DEV), a=a.to(DEV), norm_weight=w.to(DEV),
        router_weight=normal(experts, hidden).bfloat16().to(DEV), bias=normal(experts).to(DEV),
        w_in=codes(experts, 2 * inter, hidden), w_out=codes(experts, hidden, inter),
        w_in_scales=torch.full((experts, 2 * inter // 128, hidden // 128), 0.05, device=DEV),
        w_out_scales=torch.full((experts, hidden // 128, inter // 128), 0.05, device=DEV),
        grad_out=normal(bs, hidden).bfloat16().to(DEV),
        grad_ex=normal(rows, hidden).bfloat16().to(DEV),
        grad_shared=normal(bs, hidden).bfloat16().to(DEV),
        grad_residual=grad_residual.to(DEV))
    exec(compile(block("A served layer, and its gradient"), "README.md", "exec"), names)
    z = ref.bf16_sum(a, residual)
    assert torch.equal(names["z"].residual_out.cpu(), z)
    # What the last line is given, and what it makes of it.
    want, want_w, bound, mag = ref.norm_backward(names["grad_x"].cpu(), z, w, 1e-6, grad_residual)
    assert ((names["grad_h"].cpu().double() - want).abs()
            <= UBF16 * want.abs() + bound * 1.01).all()
    assert ((names["grad_norm"].cpu().double() - want_w).abs()
            <= (ref.NORM_ERROR + (2 + bs + 512) * ref.U32) * mag).all()
    assert names["grad_router"].shape == (experts, hidden)
