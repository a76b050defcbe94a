"""Dispatch and the quantised combine on more tokens than one launch has
threads for (a grid of 2^32 threads wraps).  Rows repeat with a period, so
every token's result is known from a small batch's."""

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
E = 16
PERIOD = 4096


@pytest.fixture(scope="module")
def moe():
    import combine_moe_dispatch_layout_amd as m
    m.load_library()
    assert torch.cuda.is_available()
    return m


def tokens(bs, hidden):
    """A period of rows, and bs rows that repeat it."""
    gen = torch.Generator().manual_seed(hidden)
    base = torch.randn((PERIOD, hidden), generator=gen).to(DEV, torch.bfloat16)
    return base, base.repeat(-(-bs // PERIOD), 1)[:bs]


def repeats(rows, base):
    """Whether rows [bs, C] repeat base [PERIOD, C]."""
    whole = rows.shape[0] // PERIOD * PERIOD
    return bool((rows[:whole].view(-1, *base.shape) == base).all()) and \
        torch.equal(rows[whole:], base[:rows.shape[0] - whole])


def round_robin(bs):
    """Token t to expert t % E: its rank there is t // E."""
    t = torch.arange(bs, dtype=torch.int32, device=DEV)
    per = [(bs - e + E - 1) // E for e in range(E)]
    send = torch.tensor([0] + per, dtype=torch.int32, device=DEV).cumsum(0).int()
    return (t % E).view(bs, 1), t // E, send


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("bs,hidden,fp8", [((1 << 25) + 3, 32, False), ((1 << 24) + 3, 128, True)])
def test_dispatch_beyond_one_launch(moe, bs, hidden, fp8, fused):
    base, x = tokens(bs, hidden)
    ids, rank, send = round_robin(bs)
    slot = (send[(ids[:, 0]).long()] + rank).long()
    kind = "fp8" if fp8 else "bf16"
    if fused:
        lay, *out = moe.moe_dispatch_fused(x, ids, E, 1, out_dtype=kind, capacity_rows=bs,
                                           check=True)
        assert torch.equal(lay.expand_idx, rank) and torch.equal(lay.ep_send_counts, send)
    else:
        out = moe.moe_dispatch(x, ids, rank, send, E, out_dtype=kind, capacity_rows=bs,
                               check=True)
        out = list(out) if fp8 else [out]
    if not fp8:
        assert repeats(out[0][slot], base)
        return
    small_ids, small_rank, small_send = round_robin(PERIOD)
    codes, scales = moe.moe_dispatch(base, small_ids, small_rank, small_send, E, out_dtype="fp8",
                                     capacity_rows=PERIOD)
    at = (small_send[small_ids[:, 0].long()] + small_rank).long()
    assert repeats(out[0][slot], codes[at]) and repeats(out[1][slot], scales[at])


def test_combine_fp8_beyond_one_launch(moe):
    bs, hidden = (1 << 26) + 3, 128
    gen = torch.Generator().manual_seed(1)
    codes = torch.randint(0, 120, (PERIOD, hidden), generator=gen).to(DEV, torch.uint8)
    scales = torch.rand((PERIOD, 1), generator=gen).to(DEV)
    t = torch.arange(bs, dtype=torch.int32, device=DEV)
    ids = torch.zeros((bs, 1), dtype=torch.int32, device=DEV)
    send = torch.tensor([0, PERIOD], dtype=torch.int32, device=DEV)
    w = torch.full((bs, 1), 2.0, device=DEV)
    small = moe.moe_combine_fp8(codes, scales, ids[:PERIOD], t[:PERIOD].contiguous(), send,
                                w[:PERIOD], None, 1)
    out = torch.full((bs, hidden), -5.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_combine_fp8(codes, scales, ids, t % PERIOD, send, w, None, 1, out=out, check=True)
    assert repeats(out, small)
