"""What the 8-bit pieces of tree attention hold, enumerated on the CPU with torch's conversions: a query's element as
the sum of two e4m3 numbers, and a weight as the sum of three e5m2 numbers taken from half precision."""
import numpy as np
import torch


def _bf16(lo, hi):
    """Every positive bf16 number in [lo, hi)."""
    bits = torch.arange(1, 0x7F80, dtype=torch.int32).to(torch.int16)
    x = bits.view(torch.bfloat16).float()
    return x[(x >= lo) & (x < hi)]


def test_two_e4m3_numbers_hold_a_query():
    """The row's largest element lies in [128, 256).  Exact down to 2^-2 (2^-9 of 128); below, off by at most 2^-10
    (2^-17 of 128), and not exact for some."""
    x = _bf16(2.0 ** -30, 256.0)
    first = x.to(torch.float8_e4m3fn).float()
    both = first + (x - first).to(torch.float8_e4m3fn).float()
    off = (both.double() - x.double()).abs()
    assert (off[x >= 2.0 ** -2] == 0).all()
    assert (off <= 2.0 ** -10).all()
    binade = (x >= 2.0 ** -3) & (x < 2.0 ** -2)
    assert (off[binade] > 0).any() and (off[x < 2.0 ** -4] > 0).any()


def test_three_e5m2_numbers_hold_a_weight():
    """The largest weight of a segment's first tile is put at 2^10 and none passes 2^15.  Half precision is off by 2^-11
    of the weight, or by 2^-25, half of its smallest number; the pieces by 2^-9 of the weight, three times 2^-3, or by
    2^-17 (2^-27 of 2^10), half of e5m2's smallest number, where that is more."""
    w = torch.from_numpy(np.exp2(np.random.default_rng(1).uniform(-30, 15, 200000))).float()
    # a piece: a half's upper byte, rounded half up in magnitude, as the kernels take it
    rest, total = w.half(), torch.zeros_like(w).double()
    for _ in range(3):
        bits = (rest.view(torch.int16).int() & 0xFFFF) + 0x80 & 0xFF00
        bits = torch.where(bits >= 0x8000, bits - 0x10000, bits).to(torch.int16)
        piece = bits.view(torch.float16)
        total += piece.double()
        rest = (rest.float() - piece.float()).half()
    off = (total - w.double()).abs()
    rounding = torch.clamp(2.0 ** -11 * w.double(), min=2.0 ** -25)
    assert (off <= rounding + torch.clamp(2.0 ** -9 * w.double(), min=2.0 ** -17)).all()
