"""Plain 64-bit forms of the experts' products, and their inputs, for the
tests.  Written from the formulas of include/moe_dispatch.h; nothing of the
library is used.  All on the CPU."""

import numpy as np
import torch

BLOCK = 128
SENTINEL_OUT = -12345.0          # exact in bf16
SENTINEL_CODE = 0x2A
SENTINEL_SCALE = -3.0


def values(codes):
    """float64 values of e4m3fn codes (uint8 tensor)."""
    return codes.cpu().view(torch.float8_e4m3fn).to(torch.float64)


def segments(counts, align):
    """ep_send_counts [E+1] of the padded layout."""
    padded = [(c + align - 1) // align * align for c in counts]
    return np.concatenate([[0], np.cumsum(padded)]).astype(np.int32)


def random_codes(gen, shape, spread=1.0):
    """Codes of N(0, spread) values scaled to use e4m3's range."""
    v = torch.randn(shape, generator=gen, dtype=torch.float32) * (100.0 * spread)
    return v.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def small_codes(gen, shape):
    """Codes of whole numbers from -2 to 2: sums of their products are exact."""
    v = torch.randint(-2, 3, shape, generator=gen).to(torch.float32)
    return v.to(torch.float8_e4m3fn).view(torch.uint8)


def random_scales(gen, shape):
    return torch.rand(shape, generator=gen, dtype=torch.float32) * 0.019 + 0.001


def power_scales(gen, shape):
    """1/4, 1/2, 1, 2: exact factors."""
    return torch.pow(2.0, torch.randint(-2, 2, shape, generator=gen).float())


def dequantised(codes, scales):
    """codes [.., R, C] with a scale per 128 columns of each row."""
    return values(codes) * scales.cpu().double().repeat_interleave(BLOCK, -1)


def weight_values(codes, scales):
    """codes [E, N, C] with scales [E, ceil(N/128), C/128]."""
    n = codes.shape[1]
    s = scales.cpu().double().repeat_interleave(BLOCK, 1)[:, :n].repeat_interleave(BLOCK, 2)
    return values(codes) * s


def product(x, w, counts, send):
    """(y, magnitude) in float64: y[r] = w[e] @ x[r] on the experts' rows and
    the sum of the terms' magnitudes, zero elsewhere."""
    y = torch.zeros((x.shape[0], w.shape[1]), dtype=torch.float64)
    mag = torch.zeros_like(y)
    for e, c in enumerate(counts):
        lo, hi = int(send[e]), int(send[e]) + int(c)
        y[lo:hi] = x[lo:hi] @ w[e].t()
        mag[lo:hi] = x[lo:hi].abs() @ w[e].abs().t()
    return y, mag


def sum_error(channels):
    """Bound of the gated product's fp32 error as a share of the terms' summed
    magnitude: 128 additions inside a block, each off by at most one unit
    (2^-23) however the matrix unit rounds, the two scales' product (2^-24)
    and one fused multiply-add per block (2^-24 each)."""
    return 128 * 2.0 ** -23 + (1 + channels // BLOCK) * 2.0 ** -24


def e4m3_sum_error(channels):
    """The same for the e4m3 matrix instruction: it aligns each group of 8
    products to the largest and keeps 13 bits below that one's leading bit, so
    each of the 7 others loses less than 2^-13 of the largest, which is at
    most the group's summed magnitude."""
    return 7 * 2.0 ** -13 + sum_error(channels)


def real_rows(cap, counts, send):
    mask = torch.zeros(cap, dtype=torch.bool)
    for e, c in enumerate(counts):
        mask[int(send[e]):int(send[e]) + int(c)] = True
    return mask
