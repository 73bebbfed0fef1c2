"""Attention where the plan does share a group's leading keys (it declines where sharing would
save little): each test asks the plan itself. Bounds and plain form as in
test_gpu_attn_layer.py."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_14_gb300 as gdn
from tests.test_gpu_attn_layer import BF, HF, Cache, i32

pytestmark = pytest.mark.gpu


def plan_head(c):
    """(items, items of groups, rows that joined, pieces of the groups' items)."""
    return c.plan_buf[:16].view(torch.int32).tolist()


def check_shared(c, joined=None):
    o, z = c.attn()
    c.check(o, z)
    items, of_groups, rows, pieces = plan_head(c)
    assert of_groups > 0 and rows > 0, "nothing was shared"
    if joined is not None:
        assert rows == joined
    again, y = c.attn()
    assert torch.equal(o, again) and torch.equal(z, y)
    return items, of_groups, rows, pieces


def members(rng, base, n, kinds):
    """n requests behind `base` shared tokens: rows drawn from `kinds`, some tokens of their own."""
    rows = rng.choice(kinds, n)
    return rows, base + rows + rng.integers(0, 200, n)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("D,G,ps", [(64, 4, 64), (64, 6, 16), (128, 6, 64), (128, 16, 32),
                                    (128, 1, 256), (256, 8, 16), (256, 3, 128), (256, 48, 64)])
def test_several_groups(D, G, ps, dt):
    """Three groups apart, with prompts and empty requests inside them, one member that sees fewer
    of the declared pages, requests of no group before, between and behind."""
    rng = np.random.default_rng(D + G)
    Hkv = max(1, min(4, 64 // G))
    lone = ([1, 3, 1], [77, 40, 513])
    rows, kv, groups, joined = [], [], [], 0
    for i, base in enumerate((1536, 768, 1536)):
        rows += lone[0][i:i + 1]
        kv += lone[1][i:i + 1]
        n = 40 if D < 256 else 30
        r, k = members(rng, base, n, [1, 1, 2, 3])
        r[5], k[5] = 0, base           # empty
        r[7], k[7] = 150, base + 150   # a prompt: reads the shared keys by itself
        if i == 2:
            r[9], k[9] = 1, base - 100  # limits the group to the pages that it sees
        groups.append((len(rows), n, base // ps))
        rows += r.tolist()
        kv += k.tolist()
        joined += int(r[r <= 64 // G].sum())
    c = Cache(rows, kv, Hkv * G, Hkv, D, ps, dt, groups=groups, seed=D + G)
    check_shared(c, joined)


@pytest.mark.parametrize("D,G,dt", [(64, 6, HF), (128, 6, BF), (256, 6, BF), (128, 5, HF)])
def test_heads_of_a_row_in_two_tiles(D, G, dt):
    """One group of more than 128 (row, head) pairs whose heads do not divide a tile."""
    rng = np.random.default_rng(G)
    rows, kv = members(rng, 2048, 70, [1, 2, 4, 8])
    c = Cache(rows, kv, 4 * G, 4, D, 64, dt, groups=[(0, 70, 32)], seed=3)
    _, of_groups, n, pieces = check_shared(c, int(rows.sum()))
    assert n * G > 128 and pieces > of_groups * 4  # several tiles, and cut along the keys


@pytest.mark.parametrize("D,dt", [(64, BF), (128, HF), (256, BF)])
def test_items_of_groups_that_stay_whole(D, dt):
    """Many small groups (more than a block has warps): each one's shared keys are one piece."""
    rng = np.random.default_rng(D)
    rows, kv, groups = [], [], []
    for g in range(160):
        r, k = members(rng, 128, 3, [1, 2])
        groups.append((len(rows), 3, 128 // 32))
        rows += r.tolist()
        kv += k.tolist()
    c = Cache(rows, kv, 16, 8, D, 32, dt, groups=groups, seed=D)
    _, of_groups, _, pieces = check_shared(c, sum(rows))
    assert of_groups == 160 and pieces == of_groups * 8


def test_more_requests_than_the_plan_has_threads():
    rng = np.random.default_rng(1)
    rows, kv, groups = [1, 0, 2], [30, 0, 400], []
    for g in range(40):
        r, k = members(rng, 256, 30, [0, 1, 1, 2])
        groups.append((len(rows), 30, 4))
        rows += r.tolist()
        kv += k.tolist()
    c = Cache(rows, kv, 4, 2, 64, 64, groups=groups, seed=1)
    check_shared(c, sum(rows[3:]))


def test_shared_pages_that_end_inside_a_tile():
    """Pages of 16 tokens: the shared keys end at every quarter of a tile of 64."""
    for pages in (65, 66, 67):
        rows, kv = members(np.random.default_rng(pages), pages * 16, 60, [1, 2])
        c = Cache(rows, kv, 16, 4, 128, 16, groups=[(0, 60, pages)], seed=pages)
        check_shared(c, int(rows.sum()))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_slots_without_a_token_stay_out(D):
    """NaN in every slot that holds no token, behind shared keys too."""
    rows, kv = members(np.random.default_rng(D), 96, 100, [1, 2])
    c = Cache(rows, kv, 32, 8, D, 32, groups=[(0, 100, 3)], seed=D, fill="poison")
    check_shared(c, int(rows.sum()))


def test_a_replayed_step_shares_by_its_lengths():
    """Plan and attention captured once; the lengths then change which pages are shared."""
    rows, kv = [1] * 60, [2048 + 64 + r for r in range(60)]
    c = Cache(rows, kv, 16, 4, 128, 64, groups=[(0, 60, 32)], seed=9)
    o, z = c.attn()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_attn_plan(c.dims, c.batch, c.plan_buf, c.plan_buf.numel(), c.status)
        gdn.gdn_attn(c.dims, c.batch, c.plan_buf, c.q, c.k, c.v, o, z, c.ws, c.ws.numel(),
                     c.status)
    for less in (0, 700, 1900, 3):
        c.kv = np.asarray(kv) - less * (np.arange(60) % 3)
        c.kv = np.maximum(c.kv, 1)
        c.keep[2].copy_(i32(c.kv))
        o.fill_(7)
        graph.replay()
        c.check(o, z)
        if less in (0, 3):
            assert plan_head(c)[1] > 0
