"""gdn_kv_append over row maps in which one request is bad, rows belong to several requests, or
requests are many: every good request is appended whole and its query rows are rotated, whatever
stands beside it. Most maps here have a few long requests among many short ones, which the call
serves with blocks that look their request up."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_14_gb300 as gdn
from tests.test_gpu_attn_layer import BF, check_rotated, i32, rope_inputs, rotate64

pytestmark = pytest.mark.gpu

BAD_ROWS = gdn.CODES["GDN_DEV_BAD_ROWS"]


def append(start, rows, kv, num_rows, max_rows, good, Hq=32, Hkv=8, D=128, ps=64, width=None,
           with_q=True):
    """Append with these maps; returns the status word after checking that exactly the rows of the
    `good` requests are in the cache, and rotated in q_out."""
    R = len(rows)
    g, pos, freq, axis = rope_inputs(num_rows, D, D, 1, R, 1 << 16)
    q, k, v = (torch.randn(num_rows, h, D, generator=g, device="cuda").to(BF)
               for h in (Hq, Hkv, Hkv))
    width = width or max(-(-int(kv[r]) // ps) for r in good)
    table = i32(np.random.default_rng(R).permutation(R * width).reshape(R, width))
    kc, vc = (torch.full((R * width, Hkv, ps, D), 9.0, dtype=BF, device="cuda") for _ in range(2))
    dims = gdn.make_attn_dims(Hq, Hkv, D, ps)
    maps = [i32(start), i32(rows), i32(kv)]
    batch = gdn.make_kv_batch(R, num_rows, max_rows, R * width, *maps, table)
    rope = gdn.make_rope(D, freq, pos)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.full_like(q, 9.0) if with_q else None
    gdn.gdn_kv_append(dims, batch, rope, q if with_q else None, k, v, q_out, kc, vc, status)
    code = int(status.item())
    kr, r_k = rotate64(k, pos, axis, freq, D, False, False)
    touched = torch.zeros(num_rows, dtype=torch.bool, device="cuda")
    for r in good:
        n, a = int(rows[r]), int(start[r])
        at = torch.arange(int(kv[r]) - n, int(kv[r]), device="cuda")
        page = table[r].long()[at // ps]
        check_rotated(kc[page, :, at % ps], kr[a:a + n], r_k[a:a + n])
        assert torch.equal(vc[page, :, at % ps], v[a:a + n]), r
        kc[page, :, at % ps] = 9.0
        vc[page, :, at % ps] = 9.0
        touched[a:a + n] = True
    assert bool((kc == 9).all()) and bool((vc == 9).all())  # nothing else was written
    if with_q:
        qr, r_q = rotate64(q, pos, axis, freq, D, False, False)
        check_rotated(q_out[touched], qr[touched], r_q[touched])
        assert bool((q_out[~touched] == 9).all())
    return code


def packed(rows):
    """Rows side by side: (row_start, row_len, kv_len) with some tokens before the rows."""
    rows = np.asarray(rows)
    return np.cumsum(rows) - rows, rows, rows + 7 * (np.arange(len(rows)) % 5)


@pytest.mark.parametrize("stale", ["kv_len below row_len", "row range past the rows"])
def test_a_stale_length_beside_good_requests(stale):
    """Request 0's row_len is that of an earlier step: it alone is skipped, and reported."""
    start, rows, kv = packed([0] + [1] * 39)
    rows = rows.copy()
    rows[0] = 300
    kv[0] = 20 if stale.startswith("kv") else 300
    num_rows = 339 if stale.startswith("kv") else 39
    if stale.startswith("kv"):
        start = start + 300
        start[0] = 0
    good = range(1, 40)
    assert append(start, rows, kv, num_rows, 400, good, width=8) == BAD_ROWS
    # and where the stale request is the last, and wide heads take a row a block
    rows[[0, 39]], kv[[0, 39]], start[[0, 39]] = rows[[39, 0]], kv[[39, 0]], start[[39, 0]]
    assert append(start, rows, kv, num_rows, 400, range(39), Hq=16, Hkv=2, D=256,
                  width=8) == BAD_ROWS


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 32, 8), (64, 2, 1)])
def test_rows_of_several_requests(D, Hq, Hkv):
    """Several requests continue with the same rows (samples forked from one prompt): each
    gets them in its own pages."""
    start, rows, kv = packed([300] + [1] * 38)
    start, rows = np.append(start, [0, 0]), np.append(rows, [300, 300])
    kv = np.append(kv, [310, 300])
    assert append(start, rows, kv, 338, 300, range(41), Hq=Hq, Hkv=Hkv, D=D) == 0
    start, rows, kv = np.zeros(9, int), np.full(9, 200), 200 + np.arange(9)
    rows[3:] = 1
    assert append(start, rows, kv, 200, 400, range(9), Hq=Hq, Hkv=Hkv, D=D) == 0


@pytest.mark.parametrize("where", ["first", "last", "spread"])
def test_rows_of_several_among_many_requests(where):
    """Twenty of 300 requests on the same 300 rows: several times as many blocks as rows."""
    rows = np.ones(300, int)
    long = {"first": np.arange(20), "last": np.arange(280, 300),
            "spread": np.arange(20) * 14 + 3}[where]
    rows[long] = 300
    start = np.full(300, 300)
    start[long] = 0
    short = np.setdiff1d(np.arange(300), long)
    start[short] = 300 + np.arange(280)
    kv = rows + np.arange(300) % 7
    assert append(start, rows, kv, 580, 300, range(300), Hq=4, Hkv=2) == 0
    kv[short[5]], kv[long[3]] = 0, 299  # and two bad ones among them
    good = [r for r in range(300) if r not in (short[5], long[3])]
    assert append(start, rows, kv, 580, 300, good, Hq=4, Hkv=2, width=6) == BAD_ROWS


def test_no_rows_and_a_bad_length_is_reported():
    """A request without rows whose length is past its table, beside long and short ones."""
    start, rows, kv = packed([200] + [1] * 30 + [0])
    kv[31] = 1 << 20
    assert append(start, rows, kv, 230, 400, range(31), width=8) == BAD_ROWS


@pytest.mark.parametrize("R", [128, 129, 200, 1000])
def test_many_requests(R):
    """More requests than a block has threads, empty ones and bad ones among them."""
    rng = np.random.default_rng(R)
    rows = rng.integers(0, 3, R)
    rows[rng.integers(0, R, 4)] = [150, 64, 400, 33]
    start, rows, kv = packed(rows)
    good = list(range(R))
    assert append(start, rows, kv, int(rows.sum()), 400, good, Hkv=2, Hq=4, width=7) == 0
    bad = sorted(set(rng.integers(0, R, 5).tolist()))
    for r in bad:
        kv[r] = -1
    good = [r for r in good if r not in bad]
    assert append(start, rows, kv, int(rows.sum()), 400, good, Hkv=2, Hq=4, width=7) == BAD_ROWS


@pytest.mark.parametrize("R", [3, 40])
def test_a_bound_on_the_rows_at_the_end_of_32_bits(R):
    """max_rows is an upper bound: any is allowed."""
    start, rows, kv = packed([17] + [1] * (R - 1))
    for top in ((1 << 31) - 1, (1 << 31) - 8, 17):
        assert append(start, rows, kv, int(rows.sum()), top, range(R), Hq=1, Hkv=1, D=64, width=2,
                      with_q=False) == 0
