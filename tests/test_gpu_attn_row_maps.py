"""Attention over row maps in which requests claim the same packed rows: those are skipped and
reported where they are more than the pack holds, and the other requests come out as if they were
alone. Bounds and plain form as in test_gpu_attn_layer.py."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_14_gb300 as gdn
from tests.test_gpu_attn_layer import Cache, i32

pytestmark = pytest.mark.gpu

BAD_ROWS = gdn.CODES["GDN_DEV_BAD_ROWS"]


def claim(c, start, num_rows):
    """The same requests at other places of a pack of num_rows rows."""
    c.start = np.asarray(start)
    c.T = num_rows
    c.q = c.q[:num_rows].contiguous()
    c.keep[0].copy_(i32(start))
    c.batch.num_rows = num_rows


def check(c, good, code, untouched):
    o, z = c.attn()
    assert int(c.status.item()) == code
    c.status.zero_()
    c.check(o, z, requests=good)
    for a, b in untouched:
        assert bool((o[a:b] == 7).all()) and bool((z[a:b] == 7).all())
    return c.plan_buf[:16].view(torch.int32).tolist()  # items, of groups, list rows, pieces


@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_requests_on_the_same_rows_beside_a_group(D):
    """Four requests of all 2048 rows want 256 items where the pack allows 76, before two of one
    row each whose records are taken from the end of the list."""
    pages = 39
    rows = [2048] * 4 + [1, 1]
    kv = [2048] * 4 + [pages * 128 + 3, pages * 128 + 90]
    c = Cache(rows, kv, 32, 8, D, 128, groups=[(4, 2, pages)], seed=D)
    claim(c, [0, 0, 0, 0, 2048, 2049], 2050)
    head = check(c, [4, 5], BAD_ROWS, [(0, 2048)])
    assert head[1] > 0  # the group does share


def test_some_requests_share_rows_and_some_do_not():
    rows, kv = [300, 300, 41, 1, 8, 0], [400, 300, 90, 700, 8, 0]
    c = Cache(rows, kv, 8, 2, 128, 32, seed=5)
    claim(c, [0, 0, 300, 341, 342, 10], 350)
    check(c, [2, 3, 4], BAD_ROWS, [(0, 300)])
    # a part of the rows is enough
    claim(c, [0, 41, 0, 341, 342, 10], 350)
    c.rows = np.array([60, 250, 41, 1, 8, 0])
    c.keep[1].copy_(i32(c.rows))
    check(c, [3, 4], BAD_ROWS, [(0, 341)])


def test_many_requests_on_one_row():
    """More requests than the plan has threads."""
    rows, kv = [1] * 1500, [40 + r % 50 for r in range(1500)]
    c = Cache(rows, kv, 4, 1, 64, 16, seed=6)
    start = np.zeros(1500, int)
    start[[7, 1499]] = 1, 2
    claim(c, start, 3)
    check(c, [7, 1499], BAD_ROWS, [(0, 1)])


def test_rows_of_two_requests_within_the_pack():
    """Two requests on one row of a pack that has room: not looked for, the others are right."""
    rows, kv = [1, 1, 5, 1], [200, 300, 77, 50]
    c = Cache(rows, kv, 8, 2, 128, 16, seed=7)
    claim(c, [0, 0, 1, 6], 8)
    check(c, [2, 3], 0, [(7, 8)])
