"""Rotary angles at every int32 position.

The angle of the 64-bit form is exact here: position and frequency are integers times powers of
two, so their product is formed in whole numbers and divided by 2 pi to 200 bits. Tolerance as in
test_gpu_attn_layer.py: one rounding of the result and 2^-21 of the pair's length (an angle within
2^-23, its cosine and sine to a few 2^-24, two products and a sum)."""
import math
from fractions import Fraction

import pytest
import torch

import gated_deltanet_linear_14_gb300 as gdn
from tests.test_gpu_attn_layer import check_rotated, i32

pytestmark = pytest.mark.gpu


def pi_bits(bits):
    """pi * 2^bits as a whole number, by 16 atan(1/5) - 4 atan(1/239)."""
    def atan(n):
        one = 1 << (bits + 32)
        x, total, k, sign = one // n, 0, 1, 1
        while x:
            total += sign * (x // k)
            x //= n * n
            k, sign = k + 2, -sign
        return total
    return (16 * atan(5) - 4 * atan(239)) >> 32


PI = Fraction(pi_bits(200), 1 << 200)


def turn(pos, f):
    """pos * f in radians, reduced to [-pi, pi] before it is rounded to 64 bits."""
    t = Fraction(pos) * Fraction(f) / (2 * PI)
    return float((t - round(t)) * 2 * PI)


FREQ = [1.0, 0.731, 0.25, 1e-3, 1e-5, 1e-7, 2.5e-10, -0.6, 3.75, 700.5, 0.0, 2.0 ** -120]


def test_positions_of_all_int32():
    pos = [0, 1, -1, 4095, 4096, -4097, (1 << 24) - 1, (1 << 24) + 1, 16777259, 123456789,
           -98765432, (1 << 30) + 12345, (1 << 31) - 1, -(1 << 31), -(1 << 31) + 1, 2000000011]
    rd = 2 * len(FREQ)
    freq = torch.tensor(FREQ, device="cuda", dtype=torch.float32)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    q = torch.randn(len(pos), 3, rd, generator=g, device="cuda")
    out = torch.empty_like(q)
    dims = gdn.make_attn_dims(3, 3, rd, 16, io=gdn.GDN_F32)
    gdn.gdn_rope(dims, gdn.make_rope(rd, freq, i32(pos)), q, out)
    angle = torch.tensor([[turn(p, f) for f in freq.tolist()] for p in pos], dtype=torch.float64,
                         device="cuda")
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    x, y = q.double()[..., :rd // 2], q.double()[..., rd // 2:]
    r = torch.hypot(x, y)
    check_rotated(out, torch.cat((x * c - y * s, y * c + x * s), -1), torch.cat((r, r), -1))


def test_small_angles_keep_their_leading_bits():
    """(1, 0) turned by a small angle: the sine to fp32's relative accuracy, not only the length's."""
    freq = torch.tensor([1e-2, 1e-4, 1e-6, 1e-9], device="cuda")
    pos = [1, 3, -7]
    q = torch.zeros(len(pos), 1, 8, device="cuda")
    q[..., :4] = 1
    out = torch.empty_like(q)
    dims = gdn.make_attn_dims(1, 1, 8, 16, io=gdn.GDN_F32)
    gdn.gdn_rope(dims, gdn.make_rope(8, freq, i32(pos)), q, out)
    for i, p in enumerate(pos):
        for j, f in enumerate(freq.tolist()):
            want = math.sin(turn(p, f))
            assert abs(out[i, 0, 4 + j].item() - want) <= 2.0 ** -20 * abs(want), (p, f)


def test_a_frequency_that_is_not_finite_gives_nan():
    freq = torch.tensor([math.inf, math.nan, 0.5, -math.inf], device="cuda")
    q = torch.ones(2, 1, 8, device="cuda")
    out = torch.empty_like(q)
    dims = gdn.make_attn_dims(1, 1, 8, 16, io=gdn.GDN_F32)
    gdn.gdn_rope(dims, gdn.make_rope(8, freq, i32([5, 7])), q, out)
    bad = torch.isnan(out).view(2, 2, 4)
    assert bool(bad[..., [0, 1, 3]].all()) and not bool(bad[..., 2].any())
