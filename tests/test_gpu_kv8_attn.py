"""gdn_kv8_attn against 64 bits over what the codes stand for.

How far an output may be off, with A = sum p |v| / sum p:
  q in parts: each element within 2^-10 where the row's largest has 2^7, so 2^-17 of that, and
    fp32 sums of D products: ds = scale (2^-17 max|q| sum|k| + 2^-19 sum|q k|), at most for any key
    seen: p is off by 2 ds relative to the others, o by 4 ds A;
  p in parts: fp16's half step 2^-11 and the parts' rest, 2^-7 of p in bf16, 2^-11 in fp16, and
    2^-17 where the largest p has 2^10 (2^-27 of it) for small ones: R A + n 2^-27 max|v|;
  ex2 and the fp32 sums: 2^-18 A;
  the output's rounding: eps / 2 |o|.
lse: ds, 2^-20 of the largest score's and its own size, 2^-18."""
import math

import pytest
import torch

import gated_deltanet_linear_14_gb300 as gdn
from tests.kv8_util import BF, HF, Paged, i32

pytestmark = pytest.mark.gpu
REST = {BF: 2.0 ** -7 + 2.0 ** -10, HF: 2.0 ** -10}


def fill(P, seed=0, spread=0.5):
    """Random codes and exponents in all of the cache."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    for c, e in ((P.cache.k, P.cache.k_exp), (P.cache.v, P.cache.v_exp)):
        pages, h, ps, d = c.shape
        x = torch.randn(c.shape, generator=g, device="cuda")
        x = x * torch.exp(spread * torch.randn(pages, h, ps // 16, 1, 1, generator=g, device="cuda")
                          ).expand(pages, h, ps // 16, 16, 1).reshape(pages, h, ps, 1)
        top = x.view(pages, h, ps // 16, 16 * d).abs().amax(-1)
        ex = torch.ceil(torch.log2(top / 448))
        e.copy_(ex.to(torch.int8))
        c.copy_((x * torch.exp2(-ex).repeat_interleave(16, 2)[..., None]).to(c.dtype))


def planned(P, batch):
    plan, ws = (torch.empty(size(P.dims, batch), dtype=torch.uint8, device="cuda") for size in
                (gdn.gdn_kv8_attn_plan_bytes, gdn.gdn_kv8_attn_workspace_bytes))
    gdn.gdn_kv8_attn_plan(P.dims, batch, plan, plan.numel(), P.status)
    return plan, ws


def attend(P, batch, q, lse=True):
    o = torch.full(q.shape, 7.0, device="cuda", dtype=q.dtype)
    lse = torch.full(q.shape[:2], 7.0, device="cuda") if lse else None
    plan, ws = planned(P, batch)
    gdn.gdn_kv8_attn(P.dims, batch, plan, q, P.cache.codes, o, lse, ws, ws.numel(), P.status)
    return o, lse


def check(P, q, o, lse, start, lens, kv, only=None, scale=None):
    d, g = P.dims.head_dim, P.dims.num_q_heads // P.dims.num_kv_heads
    scale = scale or 1 / math.sqrt(d)
    half = torch.finfo(q.dtype).eps / 2
    for r in range(len(lens)) if only is None else only:
        m, n, a = lens[r], kv[r], start[r]
        if m == 0:
            continue
        k, v = (P.tokens(r, n, c, e)[0] for c, e in ((P.cache.k, P.cache.k_exp),
                                                     (P.cache.v, P.cache.v_exp)))
        seen = torch.arange(n, device="cuda") < (torch.arange(m, device="cuda") + n - m + 1)[:, None]
        for h in range(P.dims.num_q_heads):
            x, kh, vh = q[a:a + m, h].double(), k[:, h // g], v[:, h // g]
            s = torch.where(seen, scale * x @ kh.t(), -math.inf)
            z = torch.logsumexp(s, -1)
            p = torch.exp(s - z[:, None])
            want, A = p @ vh, p @ vh.abs()
            ds = scale * (2.0 ** -17 * x.abs().amax(-1)[:, None] * kh.abs().sum(-1)
                          + 2.0 ** -19 * x.abs() @ kh.abs().t())
            ds = torch.where(seen, ds, 0.0).amax(-1)
            peak = p.amax(-1)
            room = ((4 * ds + REST[q.dtype] + 2.0 ** -18)[:, None] * A + want.abs() * half * 1.01
                    + (n * 2.0 ** -27 * peak)[:, None] * vh.abs().amax(0)
                    + torch.finfo(q.dtype).tiny)
            off = (o[a:a + m, h].double() - want).abs()
            assert (off <= room).all(), (r, h, (off / room).max().item())
            if lse is not None:
                big = torch.where(seen, s, 0.0).abs().amax(-1)
                off = (lse[a:a + m, h].double() - z).abs()
                assert (off <= ds + 2.0 ** -20 * (big + z.abs()) + 2.0 ** -18).all(), (r, h, off.max())


def queries(P, t, dtype, seed=0, spread=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn(t, P.dims.num_q_heads, P.dims.head_dim, generator=g, device="cuda")
    return (q * torch.exp(spread * torch.randn(t, 1, 1, generator=g, device="cuda"))).to(dtype)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("hq,hkv,d,ps,lens,kv", [
    (1, 1, 64, 16, [1], [1]), (1, 1, 128, 16, [1], [1]), (1, 1, 256, 16, [1], [1]),
    (4, 2, 128, 64, [1, 1, 1], [63, 64, 65]), (4, 2, 64, 32, [1, 2, 3, 0, 5], [1, 17, 300, 4, 5]),
    (16, 2, 256, 64, [1, 8, 1], [1000, 130, 8]), (32, 8, 128, 16, [1] * 9, list(range(1, 1800, 200))),
    (8, 1, 128, 128, [40, 3], [40, 700]), (6, 2, 64, 256, [200, 1], [513, 129]),
    (5, 5, 256, 16, [70], [257]), (128, 1, 64, 16, [2, 1], [33, 31]), (12, 3, 128, 32, [129], [129]),
    (32, 8, 128, 256, [1, 1, 1], [20000, 777, 12345]), (8, 2, 64, 128, [8, 5, 8], [9000, 130, 8]),
    (16, 2, 256, 128, [2, 4], [7000, 3001]), (16, 4, 128, 16, [8, 1, 3], [5000, 4097, 3]),
    (3, 3, 256, 32, [32, 11], [4000, 32]),
    # (long prompts, which go through 16 bits)
    (8, 1, 128, 64, [150], [700]), (16, 1, 64, 16, [64, 80], [500, 80]),
    (8, 1, 256, 256, [200, 130], [200, 1000]), (16, 2, 128, 32, [1, 300, 0, 260], [900, 300, 5, 777]), (16, 1, 64, 64, [1, 1], [40000, 64])])
def test_against_64_bits(dtype, hq, hkv, d, ps, lens, kv):
    P = Paged(len(lens), max(kv), hq, hkv, d, ps, dtype, seed=d + ps)
    fill(P, seed=1)
    start = [sum(lens[:r]) for r in range(len(lens))]
    q = queries(P, sum(lens), dtype, spread=0.5)
    o, lse = attend(P, P.batch(start, lens, kv), q)
    gdn.raise_on_status(P.status)
    check(P, q, o, lse, start, lens, kv)


def test_long_and_short_in_one_step():
    """A prompt piece, verify rows and single tokens, in rows that do not follow the requests' order,
    with rows of nobody, queries as slices of a projection, and without lse."""
    lens, kv = [300, 8, 1, 1, 17], [5000, 3000, 20000, 1, 400]
    start = [40, 0, 345, 8, 9]
    P = Paged(5, max(kv), 8, 2, 128, 64, seed=3)
    fill(P)
    qkv = queries(P, 350, BF)
    wide = torch.zeros(350, 12, 128, device="cuda", dtype=BF)
    wide[:, :8] = qkv
    q = wide[:, :8]
    o, lse = attend(P, P.batch(start, lens, kv, rows=350), q)
    o2, _ = attend(P, P.batch(start, lens, kv, rows=350), q, lse=False)
    gdn.raise_on_status(P.status)
    check(P, q, o, lse, start, lens, kv)
    assert torch.equal(o, o2)
    assert (o[340:345] == 7).all() and (o[346:] == 7).all() and (o[26:40] == 7).all()
    assert (lse[340:345] == 7).all()


@pytest.mark.parametrize("dtype,d,hq,hkv,rows", [(BF, 128, 32, 8, 1), (HF, 64, 16, 4, 4),
                                                  (BF, 256, 16, 2, 1), (HF, 128, 8, 2, 8)])
def test_shared_pages(dtype, d, hq, hkv, rows):
    """Two groups behind shared pages: the same bits' worth as without declaring them."""
    R, shared, ps = 24, 2048, 32
    kv = [shared + 10 + 7 * r for r in range(R)]
    P = Paged(R, max(kv), hq, hkv, d, ps, dtype, seed=4)
    n = shared // ps
    P.table[:12, :n] = P.table[0, :n].clone()
    P.table[12:, :n] = P.table[12, :n].clone()
    fill(P)
    lens, start = [rows] * R, [rows * r for r in range(R)]
    q = queries(P, R * rows, dtype)
    groups = i32([0, 12]), i32([12, 12]), i32([n, n])
    o, lse = attend(P, P.batch(start, lens, kv, groups=groups), q)
    gdn.raise_on_status(P.status)
    check(P, q, o, lse, start, lens, kv, only=(0, 1, 11, 12, 23))


def test_exponents_of_neighbouring_blocks_far_apart():
    """Blocks whose scales differ by up to 2^60 either way, keys' and values'."""
    P = Paged(2, 300, 4, 2, 128, 16, seed=5)
    fill(P)
    g = torch.Generator(device="cuda").manual_seed(9)
    P.cache.v_exp.copy_(torch.randint(-60, 61, P.cache.v_exp.shape, generator=g, device="cuda").to(torch.int8))
    P.cache.k_exp.copy_((torch.randint(-12, 1, P.cache.k_exp.shape, generator=g, device="cuda") - 6).to(torch.int8))
    q = queries(P, 2, BF)
    o, lse = attend(P, P.batch([0, 1], [1, 1], [300, 250]), q)
    check(P, q, o, lse, [0, 1], [1, 1], [300, 250])


def test_exponents_beyond_the_range_count_as_its_end():
    P = Paged(1, 64, 2, 1, 64, 64, seed=5)
    fill(P)
    q = queries(P, 1, BF)
    P.cache.v_exp.fill_(60)
    P.cache.k_exp.fill_(-60)
    want, _ = attend(P, P.batch([0], [1], [50]), q)
    P.cache.v_exp.fill_(100)
    P.cache.k_exp.fill_(-128)
    got, _ = attend(P, P.batch([0], [1], [50]), q)
    assert torch.equal(got, want) and torch.isfinite(got).all()


@pytest.mark.parametrize("dtype", [BF, HF])
def test_small_probabilities_that_make_up_a_part_together(dtype):
    """One key far above 60 000 equal ones: what those weigh together is not lost."""
    n = 60001
    P = Paged(1, n, 1, 1, 64, 256, dtype)
    P.cache.k.copy_(torch.zeros(P.cache.k.shape, device="cuda"))
    P.cache.v.copy_(torch.ones(P.cache.v.shape, device="cuda"))
    for e in (P.cache.k_exp, P.cache.v_exp):
        e.fill_(0)
    page = int(P.table[0, 0])
    P.cache.k.view(torch.uint8)[page, 0, 0] = 0x38   # 1
    P.cache.v.view(torch.uint8)[page, 0, 0] = 0x00
    for s in (8.0, 11.0, 14.0):
        q = torch.full((1, 1, 64), s / 8, device="cuda", dtype=dtype)
        o, lse = attend(P, P.batch([0], [1], [n]), q)
        check(P, q, o, lse, [0], [1], [n])


@pytest.mark.parametrize("rows", [1, 8, 16, 40, 190])
def test_nan_codes_reach_only_the_rows_that_see_them(rows):
    """NaN in slots past the end, in a value and in a key inside the rows' own tile."""
    kv, d = 200, 128
    P = Paged(1, 256, 4 if rows < 100 else 16, 2, d, 64, seed=6)
    half = P.dims.num_q_heads // 2   # heads of the first key head
    fill(P)
    clean = P.cache.k.clone(), P.cache.v.clone()
    at = lambda j: (int(P.table[0, j // 64]), j % 64)  # noqa: E731
    for c in (P.cache.k, P.cache.v):   # the last page's slots from 200 on
        page, slot = at(200)
        c.view(torch.uint8)[page, :, slot:] = 0xFF
    q = queries(P, rows, BF)
    batch = P.batch([0], [rows], [kv])
    o, lse = attend(P, batch, q)
    check(P, q, o, lse, [0], [rows], [kv])
    page, slot = at(190)
    P.cache.v.view(torch.uint8)[page, 1, slot, 77] = 0x7F
    o2, lse2 = attend(P, batch, q)
    bad = torch.zeros_like(o, dtype=torch.bool)
    sees = torch.arange(rows, device="cuda") + kv - rows >= 190
    bad[sees, half:, 77] = True
    assert torch.equal(o2.isnan(), bad) and torch.equal(o2[~bad], o[~bad]) and torch.equal(lse, lse2)
    P.cache.v.copy_(clean[1])
    P.cache.k.view(torch.uint8)[page, 0, slot, 5] = 0xFF
    o3, lse3 = attend(P, batch, q)
    assert o3[sees][:, :half].isnan().all() and lse3[sees][:, :half].isnan().all()
    assert torch.equal(o3[~sees], o[~sees]) and torch.equal(o3[:, half:], o[:, half:])


def test_strange_queries():
    """Rows of very different size, all zeros, infinite or NaN elements: each row by itself."""
    P = Paged(1, 500, 4, 2, 128, 32, seed=7)
    fill(P)
    q = queries(P, 8, BF)
    q[0] *= 1e-30
    q[1] = 0.0
    q[2] *= 20.0
    q[3, 0, 3], q[4, 1, 4] = float("inf"), float("nan")
    lens, kv = [8], [500]
    o, lse = attend(P, P.batch([0], lens, kv), q)
    bad = torch.zeros(8, 4, dtype=torch.bool, device="cuda")
    bad[3, 0] = bad[4, 1] = True
    assert torch.equal(o.isnan().all(-1), bad) and torch.equal(o.isnan().any(-1), bad)
    assert torch.equal(lse.isnan(), bad)
    q2 = q.clone()
    q2[bad] = 1.0
    o2, lse2 = attend(P, P.batch([0], lens, kv), q2)
    assert torch.equal(o2[~bad], o[~bad])
    check(P, q2, o2, lse2, [0], lens, kv)


def test_the_callers_scale():
    P = Paged(1, 100, 2, 1, 64, 16, seed=8)
    P.dims = gdn.make_attn_dims(2, 1, 64, 16, scale=0.5)
    fill(P)
    q = queries(P, 3, BF)
    o, lse = attend(P, P.batch([0], [3], [100]), q)
    check(P, q, o, lse, [0], [3], [100], scale=0.5)


def test_bad_requests_and_pages():
    P = Paged(4, 200, 4, 2, 128, 64, seed=9)
    fill(P)
    P.table[1, 1] = 10 ** 6
    q = queries(P, 4, BF)
    good = P.batch([0, 1, 2, 3], [1, 1, 1, 1], [200, 200, 150, 3])
    o, lse = attend(P, good, q)
    assert P.status.item() == gdn.CODES["GDN_DEV_BAD_PAGE"]
    check(P, q, o, lse, [0, 1, 2, 3], [1] * 4, [200, 200, 150, 3], only=(0, 2, 3))
    P.status.zero_()
    o, lse = attend(P, P.batch([0, 9, 2, 3], [1, 1, 1, 1], [200, 50, 150, 300], rows=4), q)
    assert P.status.item() == gdn.CODES["GDN_DEV_BAD_ROWS"]
    check(P, q, o, lse, [0, 0, 2, 0], [1] * 4, [200, 0, 150, 0], only=(0, 2))
    assert (o[1] == 7).all() and (o[3] == 7).all()


def test_a_long_prompt_with_a_bad_page_beside_a_good_one():
    P = Paged(2, 400, 16, 2, 64, 32, seed=9)
    fill(P)
    P.table[0, 3] = -5
    q = queries(P, 500, BF)
    o, lse = attend(P, P.batch([0, 200], [200, 300], [400, 333]), q)
    assert P.status.item() == gdn.CODES["GDN_DEV_BAD_PAGE"]
    check(P, q, o, lse, [0, 200], [200, 300], [400, 333], only=(1,))


def test_long_prompts_behind_shared_pages():
    """Pages are brought to 16 bits once for a group, but for those that its first request has not
    (a shorter one, one without rows) or not the same, whatever is declared."""
    R, ps, lens = 7, 32, [200, 150, 190, 0, 170, 160, 150]
    kv = [1000, 900, 1100, 640, 700, 300, 1200]
    P = Paged(R, max(kv), 16, 2, 64, ps, seed=10)
    P.table[1:3, :20] = P.table[0, :20].clone()
    P.table[4, :20] = P.table[3, :20].clone()     # first: no rows
    P.table[6, :20] = P.table[5, :20].clone()     # first: 300 keys, 9 whole pages
    P.table[6, 4] = P.table[6, 25]                # not the same after all
    fill(P)
    start = [sum(lens[:r]) for r in range(R)]
    q = queries(P, sum(lens), BF)
    groups = i32([0, 3, 5]), i32([3, 2, 2]), i32([20, 20, 20])
    o, lse = attend(P, P.batch(start, lens, kv, groups=groups), q)
    gdn.raise_on_status(P.status)
    check(P, q, o, lse, start, lens, kv)


def test_fp16_prompts_take_keys_and_values_as_read_back():
    """Codes beyond 65504 count as it, as gdn_kv8_read gives them."""
    P = Paged(1, 200, 8, 1, 64, 64, HF, seed=9)
    fill(P)
    P.cache.v_exp.fill_(12)
    q = queries(P, 160, HF)
    o, _ = attend(P, P.batch([0], [160], [200]), q)
    back = torch.empty(200, 1, 64, device="cuda", dtype=HF)
    gdn.gdn_kv8_read(P.dims, P.batch([0], [200], [200]), P.cache.codes, None, back, P.status)
    gdn.raise_on_status(P.status)
    assert back.abs().max() == 65504 and torch.isfinite(o).all()
    k = P.tokens(0, 200, P.cache.k, P.cache.k_exp)[0][:, 0]
    s = q[:, 3].double() @ k.t() / 8
    s = torch.where(torch.arange(200, device="cuda") <= torch.arange(160, device="cuda")[:, None] + 40, s, -math.inf)
    p = torch.softmax(s, -1)
    want, A = p @ back[:, 0].double(), p @ back[:, 0].double().abs()
    assert ((o[:, 3].double() - want).abs() <= 2.0 ** -8 * A + 2.0 ** -10 * want.abs()).all()


def test_a_plan_for_other_counts_is_refused():
    P = Paged(2, 100, 4, 2, 128, 64, seed=9)
    fill(P)
    plan, ws = planned(P, P.batch([0], [1], [50]))
    batch = P.batch([0, 1], [1, 1], [50, 60])
    q, big = queries(P, 2, BF), torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    big[:plan.numel()] = plan
    o = torch.full_like(q, 7.0)
    ws = torch.empty(gdn.gdn_kv8_attn_workspace_bytes(P.dims, batch), dtype=torch.uint8, device="cuda")
    gdn.gdn_kv8_attn(P.dims, batch, big, q, P.cache.codes, o, None, ws, ws.numel(), P.status)
    assert P.status.item() == gdn.CODES["GDN_DEV_STALE_STEP"] and (o == 7).all()


def test_far_pages_and_the_same_bits_again():
    """Pages beyond 4 GiB of codes; the same call twice."""
    R, ps, hkv, d = 1, 256, 8, 128
    P = Paged(R, 1024, 8, hkv, d, ps, spare=17000)
    P.table[0] = torch.tensor([16900, 3, 17003, 16500], dtype=torch.int32)
    for x in P.table[0].tolist():
        for c, e in ((P.cache.k, P.cache.k_exp), (P.cache.v, P.cache.v_exp)):
            c[x] = torch.randn(hkv, ps, d, device="cuda").to(c.dtype)
            e[x] = 0
    q = queries(P, 2, BF)
    o, lse = attend(P, P.batch([0], [2], [1000]), q)
    check(P, q, o, lse, [0], [2], [1000])
    o2, lse2 = attend(P, P.batch([0], [2], [1000]), q)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_a_step_captured_append_plan_attention():
    """Norm, rotation and append, the plan and the attention of a step, captured and replayed."""
    R, d, hq, hkv = 6, 128, 8, 2
    P = Paged(R, 256, hq, hkv, d, 64, seed=11)
    fill(P)
    g = torch.Generator(device="cuda").manual_seed(3)
    qkv = torch.randn(R, hq + 2 * hkv, d, generator=g, device="cuda").to(BF)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    kv_len = i32([5, 64, 65, 100, 200, 17])
    batch = gdn.make_kv_batch(R, R, 1, P.cache.num_pages, i32(range(R)), i32([1] * R), kv_len, P.table)
    pos = kv_len - 1
    norm = gdn.make_head_norm(torch.ones(d, device="cuda"), torch.ones(d, device="cuda"))
    rope = gdn.make_rope(d, torch.logspace(0, -4, d // 2, device="cuda"), pos)
    plan, ws = planned(P, batch)
    q_out, o = torch.empty(R, hq, d, device="cuda", dtype=BF), torch.empty(R, hq, d, device="cuda", dtype=BF)

    def step():
        gdn.gdn_kv8_append(P.dims, batch, norm, rope, q, k, v, q_out, P.cache.codes, P.status)
        gdn.gdn_kv8_attn_plan(P.dims, batch, plan, plan.numel(), P.status)
        gdn.gdn_kv8_attn(P.dims, batch, plan, q_out, P.cache.codes, o, None, ws, ws.numel(), P.status)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in range(3):
        kv_len += 1
        pos += 1
        qkv.copy_(qkv.flip(0))
        graph.replay()
        gdn.raise_on_status(P.status)
        check(P, q_out, o, None, list(range(R)), [1] * R, kv_len.tolist())


@pytest.mark.parametrize("lens,kv", [([1] * 6, [700] * 6), ([9] * 6, [700, 9, 64, 128, 300, 30]),
                                     ([300] * 2, [700, 333])])
def test_two_calls_at_once(lens, kv):
    """The same step on two streams with caches and workspaces of their own, as one after the other."""
    start = [sum(lens[:r]) for r in range(len(lens))]
    made = []
    for seed in range(2):
        P = Paged(len(lens), max(kv), 16, 4, 128, 32, seed=seed)
        fill(P, seed=seed)
        batch, q = P.batch(start, lens, kv), queries(P, sum(lens), BF, seed=seed)
        plan, ws = planned(P, batch)
        made.append((P, batch, q, plan, ws, [torch.empty_like(q) for _ in range(2)], torch.cuda.Stream()))

    def run(m, out, stream):
        P, batch, q, plan, ws = m[:5]
        for _ in range(5):
            gdn.gdn_kv8_attn(P.dims, batch, plan, q, P.cache.codes, m[5][out], None, ws, ws.numel(),
                             P.status, stream=stream)

    for m in made:
        run(m, 0, None)
    torch.cuda.synchronize()
    for m in made:
        run(m, 1, m[6])
    torch.cuda.synchronize()
    for m in made:
        gdn.raise_on_status(m[0].status)
        assert torch.equal(*m[5])


def test_requests_without_rows_or_keys():
    lens, kv = [0, 1, 0, 2], [0, 1, 40, 2]
    P = Paged(4, 48, 4, 2, 64, 16, seed=12)
    fill(P)
    q = queries(P, 5, BF)
    o, lse = attend(P, P.batch([0, 0, 1, 1], lens, kv, rows=5), q)
    gdn.raise_on_status(P.status)
    check(P, q, o, lse, [0, 0, 1, 1], lens, kv)
    assert (o[3:] == 7).all() and (lse[3:] == 7).all()


def test_one_very_long_history():
    """300 000 keys of one row and of a few, cut among all CTAs and joined."""
    n = 300001
    P = Paged(1, n, 8, 2, 64, 256, seed=13)
    fill(P, spread=0.2)
    for m in (1, 12):
        q = queries(P, m, BF)
        o, lse = attend(P, P.batch([0], [m], [n]), q)
        gdn.raise_on_status(P.status)
        check(P, q, o, lse, [0], [m], [n])


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("beside", [-1, 0, 1])
@pytest.mark.parametrize("rows", [1, 9])
def test_as_many_items_as_blocks(d, beside, rows):
    # (a block of threads an item, one item fewer and one more; two blocks to a
    # multiprocessor at D = 64, one at 256)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = sms * (1 if d == 256 else 2) + beside
    lens = [rows] * n
    kv = [rows + (r * 37) % 200 for r in range(n)]
    kv[n // 2] = 3000
    P = Paged(n, max(kv), 3, 1, d, 32, BF)
    fill(P, seed=7)
    start = [rows * r for r in range(n)]
    q = queries(P, rows * n, BF, seed=1)
    o, lse = attend(P, P.batch(start, lens, kv), q)
    gdn.raise_on_status(P.status)
    check(P, q, o, lse, start, lens, kv)


@pytest.mark.parametrize("n", [1, 63, 64, 65, 128, 129, 192, 193, 511, 1537, 6000, 48000])
@pytest.mark.parametrize("rows", [1, 40])
def test_one_request_over_all_blocks(n, rows):
    rows = min(n, rows)
    P = Paged(1, n, 8, 2, 128, 64, BF)
    fill(P, seed=n)
    q = queries(P, rows, BF, seed=2)
    o, lse = attend(P, P.batch([0], [rows], [n]), q)
    gdn.raise_on_status(P.status)
    check(P, q, o, lse, [0], [rows], [n])


@pytest.mark.parametrize("dtype", [BF, HF])
def test_few_rows_in_a_large_buffer(dtype):
    """What a request can have counts, not the buffer: nothing is brought to 16 bits."""
    P = Paged(2, 700, 16, 2, 128, 32, dtype, seed=3)
    fill(P)
    batch = P.batch([0, 1], [1, 3], [700, 200], rows=2048, max_rows=3)
    assert (gdn.gdn_kv8_attn_workspace_bytes(P.dims, batch)
            == gdn.gdn_attn_workspace_bytes(P.dims, batch))
    q = queries(P, 2048, dtype)
    o, lse = attend(P, batch, q)
    gdn.raise_on_status(P.status)
    check(P, q, o, lse, [0, 1], [1, 3], [700, 200])
    assert (o[4:] == 7).all() and (lse[4:] == 7).all()


@pytest.mark.parametrize("dtype", [BF, HF])
def test_a_long_prompt_without_room_for_copies(dtype):
    """Its step goes over the codes, and nothing is written past the workspace."""
    lens, kv = [300, 200], [700, 200]
    P = Paged(2, 700, 16, 2, 128, 32, dtype, seed=3)
    fill(P)
    batch, q = P.batch([0, 300], lens, kv), queries(P, 500, dtype)
    plan, ws = planned(P, batch)
    least = gdn.gdn_attn_workspace_bytes(P.dims, batch)
    for size in (least, ws.numel() - 1):
        store = torch.full((size + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
        o, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
        gdn.gdn_kv8_attn(P.dims, batch, plan, q, P.cache.codes, o, lse, store, size, P.status)
        gdn.raise_on_status(P.status)
        check(P, q, o, lse, [0, 300], lens, kv)
        assert (store[least:] == 0x5A).all()


# Steps for each of the kernels, 8 query and 2 key heads: few pairs as columns; 128 pairs as rows, of
# which an item fills a quarter, half or all (so many threads cut a row of q); groups that share; long
# prompts through 16 bits.
KINDS = ["one", "few", "quarter", "half", "whole", "shared", "widened"]


def step_of(kind, d=128, dtype=BF, seed=0, ps=32, scale=0.0):
    """(cache, batch, starts, rows, lengths) of a step of this kind."""
    rows = {"one": 1, "few": 3, "quarter": 7, "half": 16, "whole": 40, "shared": 2, "widened": 300}[kind]
    R, shared = (20, 1024) if kind == "shared" else (2, 0)
    lens = [rows] * R
    kv = [shared + rows + 211 + (37 * r) % 100 for r in range(R)]
    P = Paged(R, max(kv), 8, 2, d, ps, dtype, seed=seed)
    P.dims = gdn.make_attn_dims(8, 2, d, ps, io=P.dims.io_dtype, scale=scale)
    fill(P, seed=seed)
    n = shared // ps
    P.table[:, :n] = P.table[0, :n].clone()
    start = [rows * r for r in range(R)]
    groups = (i32([0]), i32([R]), i32([n])) if shared else ()
    return P, P.batch(start, lens, kv, groups=groups), start, lens, kv


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (HF, 128), (BF, 256), (HF, 256)])
@pytest.mark.parametrize("apart", [0, 5, 10, 50])
def test_exponents_apart_in_every_kernel(kind, dtype, d, apart):
    """Blocks whose scales differ by up to 2^apart either way, values and (up to 2^12) keys. In fp16
    the values stay below 448, for the outputs' sake, and a step that is brought to 16 bits holds
    what fp16 does."""
    if kind == "widened" and dtype is HF and apart > 0:
        pytest.skip("values beyond fp16's normal range")
    P, batch, start, lens, kv = step_of(kind, d, dtype, seed=apart)
    g = torch.Generator(device="cuda").manual_seed(apart)
    top = apart if dtype is BF else 0

    def between(e, lo, hi):
        return torch.randint(max(lo, -60), hi + 1, e.shape, generator=g, device="cuda").to(torch.int8)

    if apart:
        P.cache.v_exp.copy_(between(P.cache.v_exp, top - 2 * apart, top))
        P.cache.k_exp.copy_(between(P.cache.k_exp, -min(apart, 12) - 6, -6))
    q = queries(P, sum(lens), dtype, seed=apart, spread=0.3)
    o, lse = attend(P, batch, q)
    gdn.raise_on_status(P.status)
    check(P, q, o, lse, start, lens, kv, only=(0, 1, len(lens) - 1))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("end,beyond,size", [((-60, 60), (-128, 127), 1.0),
                                             ((60, -60), (61, -61), 2.0 ** -66)])
def test_exponents_beyond_the_range_in_every_kernel(kind, end, beyond, size):
    P, batch, start, lens, kv = step_of(kind)
    q = (queries(P, sum(lens), BF).float() * size).to(BF)
    got = []
    for k_exp, v_exp in (end, beyond):
        P.cache.k_exp.fill_(k_exp)
        P.cache.v_exp.fill_(v_exp)
        got.append(attend(P, batch, q))
    gdn.raise_on_status(P.status)
    (o, lse), (o2, lse2) = got
    assert torch.isfinite(o).all() and torch.isfinite(lse).all() and (o != 0).any()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_strange_queries_in_every_kernel(kind, dtype):
    """Small, zero, large, infinite and NaN rows beside one another, and one with an outlier: each
    by itself."""
    P, batch, start, lens, kv = step_of(kind, dtype=dtype)
    t = sum(lens)
    q = queries(P, t, dtype)
    bad = torch.zeros(t, 8, dtype=torch.bool, device="cuda")
    for r in {0, t // 2, t - 1}:
        q[r, 0] *= 1e-30 if dtype is BF else 1e-6
        q[r, 1] = 0.0
        q[r, 2] *= 20.0
        q[r, 3, 3], q[r, 4, 4] = float("inf"), float("nan")
        q[r, 5, 5] = 60.0
        bad[r, 3] = bad[r, 4] = True
    o, lse = attend(P, batch, q)
    assert torch.equal(o.isnan().all(-1), bad) and torch.equal(o.isnan().any(-1), bad)
    assert torch.equal(lse.isnan(), bad)
    q2 = q.clone()
    q2[bad] = 1.0
    o2, lse2 = attend(P, batch, q2)
    gdn.raise_on_status(P.status)
    assert torch.equal(o2[~bad], o[~bad]) and torch.equal(lse2[~bad], lse[~bad])
    check(P, q2, o2, lse2, start, lens, kv, only=(0, len(lens) // 2, len(lens) - 1))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("rows", [1, 3, 7, 40, 300])
def test_small_probabilities_in_every_kernel(dtype, rows):
    """One key far above 20 000 equal ones, as in the test of a single row."""
    n = 20001
    P = Paged(1, n, 8, 2, 64, 256, dtype)
    P.cache.k.copy_(torch.zeros(P.cache.k.shape, device="cuda"))
    P.cache.v.copy_(torch.ones(P.cache.v.shape, device="cuda"))
    for e in (P.cache.k_exp, P.cache.v_exp):
        e.fill_(0)
    page = int(P.table[0, 0])
    P.cache.k.view(torch.uint8)[page, :, 0] = 0x38   # 1
    P.cache.v.view(torch.uint8)[page, :, 0] = 0x00
    for s in (8.0, 14.0):
        q = torch.full((rows, 8, 64), s / 8, device="cuda", dtype=dtype)
        o, lse = attend(P, P.batch([0], [rows], [n]), q)
        check(P, q, o, lse, [0], [rows], [n])


@pytest.mark.parametrize("kind", KINDS)
def test_the_callers_scale_in_every_kernel(kind):
    P, batch, start, lens, kv = step_of(kind, d=64, scale=0.5)
    q = queries(P, sum(lens), BF)
    o, lse = attend(P, batch, q)
    check(P, q, o, lse, start, lens, kv, only=(0, len(lens) - 1), scale=0.5)


@pytest.mark.parametrize("kind", KINDS)
def test_a_bad_page_in_every_kernel(kind):
    P, batch, start, lens, kv = step_of(kind)
    P.table[1, kv[1] // 32 - 2] = 10 ** 6   # (of its own pages)
    q = queries(P, sum(lens), BF)
    o, lse = attend(P, batch, q)
    assert P.status.item() == gdn.CODES["GDN_DEV_BAD_PAGE"]
    check(P, q, o, lse, start, lens, kv, only=[r for r in (0, 2, 19) if r < len(lens)])


@pytest.mark.parametrize("dtype", [BF, HF])
def test_nan_codes_behind_shared_pages(dtype):
    """In a shared value: that element of all rows. In a key of a request's own: its rows."""
    P, batch, start, lens, kv = step_of("shared", dtype=dtype)
    q = queries(P, sum(lens), dtype)
    o, lse = attend(P, batch, q)
    at = lambda r, j: (int(P.table[r, j // 32]), j % 32)  # noqa: E731
    page, slot = at(0, 100)
    P.cache.v.view(torch.uint8)[page, 1, slot, 77] = 0xFF
    page, slot = at(3, 1100)
    P.cache.k.view(torch.uint8)[page, 0, slot, 9] = 0x7F
    o2, lse2 = attend(P, batch, q)
    gdn.raise_on_status(P.status)
    bad = torch.zeros_like(o, dtype=torch.bool)
    bad[:, 4:, 77] = True
    bad[6:8, :4] = True
    assert torch.equal(o2.isnan(), bad) and torch.equal(o2[~bad], o[~bad])
    sees = torch.zeros_like(lse, dtype=torch.bool)
    sees[6:8, :4] = True
    assert torch.equal(lse2.isnan(), sees) and torch.equal(lse2[~sees], lse[~sees])


@pytest.mark.parametrize("rows", [1, 3, 40])
@pytest.mark.parametrize("n,bits,late", [(301, 8, True), (20001, 17, False), (20001, 17, True)])
def test_weights_of_keys_whose_values_are_far_smaller(rows, n, bits, late):
    """One key of values 2^60 among keys of values 2^-60 that weigh 2^-bits of it each, and as
    much together as it does or a part of that: the sum counts them."""
    R = 200 if rows < 40 else 40
    P = Paged(1, n, 8, 2, 64, 256)
    P.table = P.table.repeat(R, 1)   # (all requests read the same: items of many tiles)
    P.cache.k.copy_(torch.zeros(P.cache.k.shape, device="cuda"))
    P.cache.v.copy_(torch.ones(P.cache.v.shape, device="cuda"))
    P.cache.k_exp.zero_()
    P.cache.v_exp.fill_(-60)
    at = n - 50 if late else 5
    page, slot = int(P.table[0, at // 256]), at % 256
    P.cache.k.view(torch.uint8)[page, :, slot] = 0x38   # 1
    block = slot // 16
    P.cache.v_exp[page, :, block] = 60
    P.cache.v.view(torch.uint8)[page, :, 16 * block:16 * block + 16] = 0
    P.cache.v.view(torch.uint8)[page, :, slot] = 0x38
    q = torch.full((R * rows, 8, 64), bits * math.log(2) / 8, device="cuda", dtype=BF)
    start, lens, kv = [rows * r for r in range(R)], [rows] * R, [n] * R
    o, lse = attend(P, P.batch(start, lens, kv), q)
    gdn.raise_on_status(P.status)
    check(P, q, o, lse, start, lens, kv, only=(0, R // 2, R - 1))
