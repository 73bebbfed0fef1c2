"""Attention of values where the numbers are hard: probabilities far below the largest, infinite
and NaN keys and values in both types, score scales of the caller. Bounds and plain form as in
test_gpu_attn_layer.py."""
import math

import numpy as np
import pytest
import torch

import gated_deltanet_linear_14_gb300 as gdn
from tests.test_gpu_attn_layer import BF, CODE, HF, Cache, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [HF, BF])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("below", [9.0, 12.0, 17.2, 18.5])
def test_many_keys_far_below_one(D, dt, below):
    """One key takes nearly all of a row's weight (its first token, as models learn it); 200 000
    others, each e^-below of that, carry a part of the output that must not be rounded away.
    Their rounding is the same for all, so it does not average out."""
    n = 200001
    c = Cache([1, 1], [n, 300], 2, 1, D, 256, dt, seed=D)
    c.k.zero_()
    c.q.zero_()
    c.q[..., 0] = 4.0
    c.k[int(c.table[0, 0]), 0, 0, 0] = below * math.sqrt(D) / 4.0
    c.v.fill_(1.0)
    c.v[int(c.table[0, 0]), 0, 0] = 0.0
    c.check(*c.attn())


@pytest.mark.parametrize("dt", [HF, BF])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("below", [12.0, 17.2, 18.5])
def test_many_keys_far_below_one_in_whole_items(D, dt, below):
    """The same with so many requests (on the same pages) that no request's keys are cut into
    parts with maxima of their own."""
    R, n = 152, 60001
    c = Cache([1] * R, [n] + [1] * (R - 1), 2, 2, D, 256, dt, seed=D)
    c.kv[:] = n
    c.keep[2].fill_(n)
    c.table[:] = c.table[0]
    c.keep[3].copy_(i32(c.table))
    c.k.zero_()
    c.q.zero_()
    c.q[..., 0] = 4.0
    first = int(c.table[0, 0])
    c.k[first, :, 0, 0] = below * math.sqrt(D) / 4.0
    c.v.fill_(1.0)
    c.v[first, :, 0] = 0.0
    o, z = c.attn()
    c.check(o, None, requests=[0, R // 2, R - 1])
    # (a tile's sum joins the row's in fp32, n / 64 times one after the other, 2^-24 each)
    assert (z[0].double() - c.ref(0)[2]).abs().max().item() <= 2.0 ** -16 + n / 64 * 2.0 ** -24
    assert bool((o == o[0]).all()) and bool((z == z[0]).all())


@pytest.mark.parametrize("dt", [HF, BF])
@pytest.mark.parametrize("scale", [0.02, 0.3, 1.0, 0.0, -1.0])
def test_the_callers_scale(scale, dt):
    """A positive scale is taken as it is, others stand for D^-1/2."""
    c = Cache([1, 5, 70], [700, 130, 300], 8, 2, 64, 16, dt, seed=4)
    c.q.mul_(0.25)
    c.dims = gdn.make_attn_dims(8, 2, 64, 16, io=CODE[dt], scale=scale)
    s = np.float32(scale) if scale > 0 else 64 ** -0.5
    c.check(*c.attn(), q=c.q.double() * float(s) * 8.0)


@pytest.mark.parametrize("dt,D,rows,kv,bad", [
    (HF, 128, 9, 140, 135), (HF, 64, 150, 300, 200), (HF, 256, 4, 4, 2), (BF, 64, 9, 140, 135),
    (BF, 256, 150, 300, 200)])
def test_infinite_and_nan_values_stay_with_the_rows_that_see_them(dt, D, rows, kv, bad):
    c = Cache([1, rows, 1], [50, kv, 70], 4, 2, D, 16, dt, seed=9)
    p, j = c.table[1, bad // 16], bad % 16
    c.v[p, :, j, 3] = math.nan
    c.v[p, :, j, 5] = math.inf
    c.v[p, :, j, D - 1] = -math.inf
    o, z = c.attn()
    c.check(o, z, requests=[0, 2])
    blind = rows - (kv - bad)  # rows that do not see token `bad`
    ref, bound, lse = c.ref(1)
    a = int(c.start[1])
    assert bool(((o[a:a + blind].double() - ref[:blind]).abs() <= bound[:blind]).all())
    seeing = o[a + blind:a + rows]
    assert bool(torch.isnan(seeing[..., 3]).all())
    assert bool((seeing[..., 5] == math.inf).all()) and bool((seeing[..., D - 1] == -math.inf).all())
    rest = [d for d in range(D) if d not in (3, 5, D - 1)]
    assert bool(((seeing.double() - ref[blind:]).abs() <= bound[blind:])[..., rest].all())
    assert (z[a:a + rows].double() - lse).abs().max().item() <= 2.0 ** -16


@pytest.mark.parametrize("dt", [HF, BF])
def test_the_largest_finite_values(dt):
    """Values at the type's largest: the sums hold them, equal ones come out as they are."""
    top = torch.finfo(dt).max
    c = Cache([1, 40], [513, 200], 4, 2, 128, 32, dt, seed=11)
    c.v.fill_(top)
    o, _ = c.attn()
    assert int(c.status.item()) == 0
    # rounded weights may sum to a little more than their unrounded sum: then the largest rounds up
    near = o.double() / top
    assert bool((torch.isinf(o) | ((near - 1).abs() <= 2.0 ** (-7 if dt == BF else -10))).all())
