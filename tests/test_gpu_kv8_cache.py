"""The append to an 8-bit cache and reading it back, against 64-bit forms.

A stored value is its value rounded once to the grid of its block: half a grid step, and before it
what fp32 does to a key (2^-18 of its pair, see test_gpu_norm_rope.py). Values (v) see no arithmetic and
are exact. A block's exponent is the least that holds its largest value; a key's block may come out
one higher or lower only where its largest value is within 2^-18 of the limit."""
import math

import pytest
import torch

import gated_deltanet_linear_14_gb300 as gdn
from gated_deltanet_linear_14_gb300.pages import Kv8Cache
from tests.kv8_util import (BF, BLOCK, CODE, F32, HF, Blocks, Paged, grid_step, i32, least_exponent,
                            normed, partners, rotated)

pytestmark = pytest.mark.gpu


def rows_for(P, t, seed=0, spread=1.0):
    d, hq, hkv = P.dims.head_dim, P.dims.num_q_heads, P.dims.num_kv_heads
    dtype = {v: k for k, v in CODE.items()}[P.dims.io_dtype]
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(t, hq + 2 * hkv, d, generator=g, device="cuda")
    x = (x * torch.exp(spread * torch.randn(t, 1, 1, generator=g, device="cuda"))).to(dtype)
    return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("hq,hkv,d,rd,ps,axes,inter,norm_on,lens,befores", [
    (4, 2, 128, 128, 16, 1, False, True, [1], [0]),
    (4, 2, 128, 128, 64, 1, True, True, [1, 40, 3, 16], [7, 0, 30, 16]),
    (16, 2, 256, 64, 32, 3, False, True, [5, 130, 1], [11, 16, 31]),
    (2, 1, 64, 64, 256, 1, False, False, [33, 2, 300], [15, 250, 5]),
    (8, 8, 64, 32, 16, 1, True, True, [17], [47]),
    (6, 3, 256, 0, 128, 1, False, True, [20, 20], [1, 2])])
def test_append_and_read(dtype, hq, hkv, d, rd, ps, axes, inter, norm_on, lens, befores):
    R, most = len(lens), max(a + b for a, b in zip(lens, befores))
    P = Paged(R, most, hq, hkv, d, ps, dtype, seed=d)
    g = torch.Generator(device="cuda").manual_seed(1)
    qw, kw = (1 + 0.3 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    inv = (1e4 ** -(torch.arange(max(rd // 2, 1), device="cuda").double() / max(rd // 2, 1))).float()
    axis = (torch.arange(max(rd // 2, 1), device="cuda") % axes).int()
    norm = gdn.make_head_norm(qw, kw, eps=1e-6, offset=0.5) if norm_on else None
    kb, vb = ([Blocks(hkv, d) for _ in range(R)] for _ in range(2))
    # what stands before, then the step itself
    for turn, (n, at) in enumerate(((befores, [0] * R), (lens, befores))):
        t = sum(n)
        if t == 0:
            continue
        q, k, v = rows_for(P, t, seed=turn, spread=1.5 if turn else 0.5)
        pos = torch.randint(0, 100000, (axes, t), generator=g, device="cuda", dtype=torch.int32)
        rope = gdn.make_rope(rd, inv, pos, axis=axis, interleaved=inter)
        start = [sum(n[:r]) for r in range(R)]
        kv = [a + b for a, b in zip(n, at)]
        batch = P.batch(start, n, kv, rows=t)
        q_out = torch.full((t, hq, d), 7.0, device="cuda", dtype=dtype)
        with_q = norm is not None or rd > 0
        gdn.gdn_kv8_append(P.dims, batch, norm, rope, q if with_q else None, k, v,
                           q_out if with_q else None, P.cache.codes, P.status)
        gdn.raise_on_status(P.status)
        y = normed(k, kw, 1e-6, 0.5) if norm_on else k.double()
        turned = rotated(y, rd, inv, pos, axis, inter)
        room = partners(y, rd, inter) * 2.0 ** -18 if norm_on or rd else 0 * y
        if with_q:
            yq = normed(q, qw, 1e-6, 0.5) if norm_on else q.double()
            want = rotated(yq, rd, inv, pos, axis, inter)
            half = torch.finfo(dtype).eps / 2
            assert ((q_out.double() - want).abs() <= want.abs() * half * (1 + 2.0 ** -10)
                    + partners(yq, rd, inter) * 2.0 ** -18 + 1e-7).all()
        k_back, v_back = (torch.full((t, hkv, d), 7.0, device="cuda", dtype=dtype) for _ in range(2))
        gdn.gdn_kv8_read(P.dims, batch, P.cache.codes, k_back, v_back, P.status)
        for r in range(R):
            a, b = start[r], start[r] + n[r]
            if not n[r]:
                continue
            vb[r].append(v[a:b].double(), at[r])
            x, e = P.tokens(r, kv[r], P.cache.v, P.cache.v_exp)
            assert torch.equal(e, vb[r].e) and torch.equal(x, vb[r].x)
            assert torch.equal(v_back[a:b].double(), x[at[r]:])
            x, e = P.tokens(r, kv[r], P.cache.k, P.cache.k_exp)
            assert torch.equal(k_back[a:b].double(), x[at[r]:])
            kb[r].append(turned[a:b], at[r])
            new, first = turned[a:b], at[r] // BLOCK
            # exponents: equal, but for largest values next to a limit
            off = e != kb[r].e
            near = torch.zeros_like(off)
            for bl in range(first, len(e)):
                part = new[max(bl * BLOCK, at[r]) - at[r]:bl * BLOCK + BLOCK - at[r]]
                top = part.abs().amax(-1).amax(0)
                near[bl] = (least_exponent(top * (1 - 2.0 ** -18))
                            != least_exponent(top * (1 + 2.0 ** -18)))
            assert not (off & ~near).any()
            unit = torch.exp2(e.double()).repeat_interleave(BLOCK, 0)[:kv[r], :, None]
            miss = (x[at[r]:] - new).abs() - room[a:b]
            assert (miss <= grid_step(new / unit[at[r]:]) / 2 * unit[at[r]:] * (1 + 1e-9)).all()
            # older tokens: their stored values, rounded anew where the exponent grew
            if at[r] and not off.any():
                assert ((x[:at[r]] - kb[r].x[:at[r]]).abs()
                        <= grid_step(kb[r].x[:at[r]] / unit[:at[r]]) * unit[:at[r]]).all()
                same = torch.equal(x[:at[r] // BLOCK * BLOCK], kb[r].x[:at[r] // BLOCK * BLOCK]) \
                    if not (norm_on or rd) else True
                assert same
            kb[r].x, kb[r].e = x.clone(), e.clone()   # go on from what is stored


def test_tokens_one_by_one_as_all_at_once():
    """Raising a block's power of two is exact but for values that fall below 2^-6 of it: those are
    rounded twice, by at most half a step of 2^-9 each time."""
    T, d = 70, 128
    P, O = Paged(1, T, 2, 1, d, 32), Paged(1, T, 2, 1, d, 32)
    _, k, v = rows_for(P, T, spread=2.0)
    gdn.gdn_kv8_append(P.dims, P.batch([0], [T], [T]), None, None, None, k, v, None,
                       P.cache.codes, P.status)
    for t in range(T):
        gdn.gdn_kv8_append(O.dims, O.batch([0], [1], [t + 1]), None, None, None, k[t:t + 1],
                           v[t:t + 1], None, O.cache.codes, O.status)
    gdn.raise_on_status(P.status)
    gdn.raise_on_status(O.status)
    for name in "kv":
        (x, e), (y, f) = (S.tokens(0, T, getattr(S.cache, name), getattr(S.cache, name + "_exp"))
                          for S in (P, O))
        assert torch.equal(e, f)
        unit = torch.exp2(e.double()).repeat_interleave(BLOCK, 0)[:T, :, None]
        assert ((x - y).abs() <= 2.0 ** -9 * unit).all()
        big = x.abs() >= 2.0 ** -6 * unit
        assert torch.equal(x[big], y[big])


def test_a_block_begun_anew_forgets_its_scale():
    P = Paged(1, 32, 2, 1, 64, 16)
    _, k, v = rows_for(P, 16)
    for size in (1e6, 1e-6):
        batch = P.batch([0], [16], [16])
        gdn.gdn_kv8_append(P.dims, batch, None, None, None, (k * size).to(BF), (v * size).to(BF),
                           None, P.cache.codes, P.status)
        x, e = P.tokens(0, 16, P.cache.v, P.cache.v_exp)
        want = (v * size).to(BF).double()
        assert torch.equal(e, least_exponent(want.abs().amax(-1).amax(0))[None])
        assert ((x - want).abs() <= want.abs().amax() * 2.0 ** -4).all()


def test_infinite_nan_zero_and_far_values():
    P = Paged(1, 64, 2, 1, 64, 64)
    x = torch.ones(64, 1, 64, device="cuda", dtype=BF)
    x[3, 0, 5], x[4, 0, 6], x[5, 0, 7] = float("inf"), float("-inf"), float("nan")
    x[16:32] = 0.0
    x[32:48] *= 1e30       # beyond 448 2^60
    x[48:] *= 1e-30        # below 2^-69
    gdn.gdn_kv8_append(P.dims, P.batch([0], [64], [64]), None, None, None, x, -x, None,
                       P.cache.codes, P.status)
    gdn.raise_on_status(P.status)
    y, e = P.tokens(0, 64, P.cache.k, P.cache.k_exp)
    assert e[:, 0].tolist() == [-8, -60, 60, -60]
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[3, 0, 5] = bad[4, 0, 6] = bad[5, 0, 7] = True
    assert torch.equal(y.isnan(), bad) and (y[:16][~bad[:16]] == 1).all()
    assert (y[16:32] == 0).all() and (y[32:48] == 448 * 2.0 ** 60).all() and (y[48:] == 0).all()
    back = torch.empty(64, 1, 64, device="cuda", dtype=F32)
    dims = gdn.make_attn_dims(2, 1, 64, 64, io=gdn.GDN_F32)
    gdn.gdn_kv8_read(dims, P.batch([0], [64], [64]), P.cache.codes, None, back, P.status)
    assert torch.equal(back.isnan(), bad) and torch.equal(back.double()[~bad], -y[~bad])
    # fp16 holds no more than 65504
    h, dims = torch.empty(64, 1, 64, device="cuda", dtype=HF), gdn.make_attn_dims(2, 1, 64, 64, io=gdn.GDN_F16)
    gdn.gdn_kv8_read(dims, P.batch([0], [64], [64]), P.cache.codes, h, None, P.status)
    assert torch.equal(h.isnan(), bad) and (h[32:48] == 65504).all()
    # an infinite key in the norm: itself NaN, 0 beside it
    gdn.gdn_kv8_append(P.dims, P.batch([0], [16], [16]), gdn.make_head_norm(eps=1e-6), None, None,
                       x[:16], x[:16], None, P.cache.codes, P.status)
    y, _ = P.tokens(0, 16, P.cache.k, P.cache.k_exp)
    assert y[3, 0, 5].isnan() and (y[3, 0, 6:] == 0).all() and y[5].isnan().all()


def test_read_whole_histories_into_strided_rows_of_every_type():
    lens, d, hkv = [100, 1, 0, 37], 128, 3
    P = Paged(4, 100, 3, hkv, d, 32)
    _, k, v = rows_for(P, sum(lens))
    start = [0, 100, 101, 101]
    batch = P.batch(start, lens, lens)
    gdn.gdn_kv8_append(P.dims, batch, None, None, None, k, v, None, P.cache.codes, P.status)
    for dtype in (BF, HF, F32):
        dims = gdn.make_attn_dims(3, hkv, d, 32, io=CODE[dtype])
        for pad, shift in ((0, 0), (8, 0), (3, 1)):
            gap = hkv * d + pad
            store = torch.full((2, 140 * gap), 7.0, device="cuda", dtype=dtype)
            outs = [torch.as_strided(s, (140, hkv, d), (gap, d, 1), s.storage_offset() + shift)
                    for s in store[:, :].unbind(0)] if shift == 0 else \
                   [torch.as_strided(s, (139, hkv, d), (gap, d, 1), s.storage_offset() + shift)
                    for s in store.unbind(0)]
            gdn.gdn_kv8_read(dims, batch, P.cache.codes, outs[0], outs[1], P.status)
            gdn.raise_on_status(P.status)
            for r in range(4):
                if not lens[r]:
                    continue
                for out, name in zip(outs, "kv"):
                    x, _ = P.tokens(r, lens[r], getattr(P.cache, name), getattr(P.cache, name + "_exp"))
                    assert torch.equal(out[start[r]:start[r] + lens[r]], x.to(dtype))
            assert (outs[0][138] == 7).all()   # rows of no request


def test_slots_and_pages_of_others_keep_what_they_hold():
    P = Paged(2, 40, 2, 1, 64, 16)
    _, k, v = rows_for(P, 5)
    before = P.cache.k.view(torch.uint8).clone(), P.cache.k_exp.clone()
    gdn.gdn_kv8_append(P.dims, P.batch([0, 5], [5, 0], [25, 3]), None, None, None, k, v, None,
                       P.cache.codes, P.status)
    gdn.raise_on_status(P.status)
    page = int(P.table[0, 1])   # tokens 20..24 are slots 4..8 of its second page
    codes, exps = P.cache.k.view(torch.uint8).clone(), P.cache.k_exp.clone()
    assert (codes[page, :, 9:] == before[0][page, :, 9:]).all()
    codes[page], exps[page] = before[0][page], before[1][page]
    assert torch.equal(codes, before[0]) and torch.equal(exps, before[1])


def test_bad_requests_and_pages_are_skipped_and_reported():
    P = Paged(4, 48, 2, 1, 64, 16, spare=0)
    _, k, v = rows_for(P, 20)
    P.table[1, 0] = 99
    P.table[3, 1] = -1
    # request 0: rows outside; 1: a bad first page; 2: longer than the table; 3: a bad second page
    batch = P.batch([18, 0, 0, 0], [5, 5, 5, 20], [5, 5, 50, 20], rows=20)
    back = torch.full((20, 1, 64), 7.0, device="cuda", dtype=BF)
    gdn.gdn_kv8_append(P.dims, batch, None, None, None, k, v, None, P.cache.codes, P.status)
    assert P.status.item() in (gdn.CODES["GDN_DEV_BAD_ROWS"], gdn.CODES["GDN_DEV_BAD_PAGE"])
    P.status.zero_()
    gdn.gdn_kv8_read(P.dims, batch, P.cache.codes, None, back, P.status)
    assert P.status.item() in (gdn.CODES["GDN_DEV_BAD_ROWS"], gdn.CODES["GDN_DEV_BAD_PAGE"])
    assert (back[16:] == 7).all() and not (back[:16] == 7).all(-1).any()
    codes = P.cache.k.view(torch.uint8)
    page = int(P.table[3, 0])
    assert (codes[page] != 0x7F).all()
    codes[page] = 0x7F
    assert (codes == 0x7F).all()


def test_several_requests_continue_with_the_same_rows():
    """More rows than there are: every request gets them in its own pages, however the grid is made."""
    R, T = 300, 40
    P = Paged(R, T, 2, 1, 64, 16)
    _, k, v = rows_for(P, T)
    for lens in ([T] * R, [1] * (R - 1) + [T]):
        batch = P.batch([0] * R, lens, lens, rows=T)
        gdn.gdn_kv8_append(P.dims, batch, None, None, None, k, v, None, P.cache.codes, P.status)
        gdn.raise_on_status(P.status)
        for r in (0, 1, R // 2, R - 2, R - 1):
            want = Blocks(1, 64)
            want.append(v[:lens[r]].double(), 0)
            x, _ = P.tokens(r, lens[r], P.cache.v, P.cache.v_exp)
            assert torch.equal(x, want.x)


@pytest.mark.parametrize("R,long", [(200, 3000), (1, 5000), (5000, 1)])
def test_many_requests_beside_a_long_one(R, long):
    lens = [1] * R
    lens[R // 2] = long
    P = Paged(R, long, 2, 1, 64, 256, spare=0) if R * long < 4e6 else None
    start = [sum(lens[:r]) for r in range(R)] if R < 1000 else list(range(R))
    _, k, v = rows_for(P, sum(lens))
    batch = P.batch(start, lens, lens)
    gdn.gdn_kv8_append(P.dims, batch, None, None, None, k, v, None, P.cache.codes, P.status)
    back = torch.empty(sum(lens), 1, 64, device="cuda", dtype=BF)
    gdn.gdn_kv8_read(P.dims, batch, P.cache.codes, None, back, P.status)
    gdn.raise_on_status(P.status)
    for r in (0, R // 2, R - 1):
        want = Blocks(1, 64)
        want.append(v[start[r]:start[r] + lens[r]].double(), 0)
        assert torch.equal(back[start[r]:start[r] + lens[r]].double(), want.x)


def test_pages_beyond_4_gib():
    hkv, d, ps, pages = 8, 128, 256, 17000     # 4.46e9 bytes of keys
    dims = gdn.make_attn_dims(8, hkv, d, ps)
    cache = Kv8Cache(dims, pages)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = torch.randn(300, hkv, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(0)).to(BF)
    batch = gdn.make_kv_batch(1, 300, 300, pages, i32([0]), i32([300]), i32([300]),
                              i32([pages - 1, 16500]).view(1, 2))
    gdn.gdn_kv8_append(dims, batch, None, None, None, x, x, None, cache.codes, status)
    back = torch.empty_like(x), torch.empty_like(x)
    gdn.gdn_kv8_read(dims, batch, cache.codes, *back, status)
    gdn.raise_on_status(status)
    want = Blocks(hkv, d)
    want.append(x.double(), 0)
    assert torch.equal(back[0].double(), want.x) and torch.equal(back[1].double(), want.x)


def test_captured_and_replayed_on_two_streams():
    """Two captured steps on caches of their own, replayed at once."""
    made = []
    for seed in range(2):
        P = Paged(8, 64, 4, 2, 128, 16, seed=seed)
        _, k, v = rows_for(P, 8 * 20, seed=seed)
        batch = P.batch(range(0, 160, 20), [20] * 8, [33] * 8)
        back = torch.empty(160, 2, 128, device="cuda", dtype=BF)

        def step(P=P, k=k, v=v, batch=batch, back=back):
            gdn.gdn_kv8_append(P.dims, batch, None, None, None, k, v, None, P.cache.codes, P.status)
            gdn.gdn_kv8_read(P.dims, batch, P.cache.codes, None, back, P.status)

        P.cache.v_exp.fill_(-60)
        P.cache.k_exp.fill_(-60)
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        k.copy_(k.flip(0)), v.copy_(v.flip(0))
        made.append((P, v, back, graph, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _, _, _, graph, stream in made:
        with torch.cuda.stream(stream):
            graph.replay()
    torch.cuda.synchronize()
    for P, v, back, _, _ in made:
        gdn.raise_on_status(P.status)
        # (the first block of a request keeps the larger of its exponents)
        assert ((back - v).abs().double() <= v.abs().amax().double() * 2.0 ** -4).all()
        x, _ = P.tokens(3, 33, P.cache.v, P.cache.v_exp)
        assert torch.equal(back[60:80].double(), x[13:])


@pytest.mark.parametrize("norm_on", [True, False])
def test_keys_next_to_the_middle_of_two_codes_come_to_the_right_one(norm_on):
    """Codes of keys as a rounding of the 64-bit values gives them: of 2 million keys dozens lie within
    4 ulp of the middle between two codes (8 of the 2^20 ulp from one middle to the next), where
    fp32 may err. Not counted: keys smaller than the other of their pair (a turn errs by ulp of
    |x| + |y|, c = (|x| + |y|) / |x| times as many of x's own: at c > 2 more than the 4) and keys below
    2^-5 of their block's scale, which are left to the fp32 value; all are held to half a step
    and 2^-18 of the pair by test_append_and_read."""
    T, d, hkv = 4096, 128, 4
    P = Paged(1, T, 4, hkv, d, 64, seed=21)
    _, k, v = rows_for(P, T, seed=4, spread=0.3)
    g = torch.Generator(device="cuda").manual_seed(5)
    kw = 1 + 0.3 * torch.randn(d, generator=g, device="cuda")
    inv = (1e4 ** -(torch.arange(d // 2, device="cuda").double() / (d // 2))).float()
    pos = torch.arange(7, T + 7, device="cuda", dtype=torch.int32)
    norm = gdn.make_head_norm(None, kw, eps=1e-6) if norm_on else None
    gdn.gdn_kv8_append(P.dims, P.batch([0], [T], [T]), norm, gdn.make_rope(d, inv, pos), None, k, v,
                       None, P.cache.codes, P.status)
    gdn.raise_on_status(P.status)
    y = normed(k, kw, 1e-6, 0.0) if norm_on else k.double()
    turned = rotated(y, d, inv, pos)
    want = Blocks(hkv, d)
    want.append(turned, 0)
    x, e = P.tokens(0, T, P.cache.k, P.cache.k_exp)
    larger = turned.abs() >= turned.roll(d // 2, -1).abs()
    same = (e == want.e).repeat_interleave(BLOCK, 0)[..., None]
    unit = torch.exp2(e.double()).repeat_interleave(BLOCK, 0)[..., None]
    counted = same & larger & (want.x.abs() >= 2.0 ** -5 * unit)
    assert counted.sum() > 10 ** 6 and not ((x != want.x) & counted).any()


def test_query_rows_of_no_request_keep_what_they_hold():
    P = Paged(2, 40, 4, 2, 128, 16)
    q, k, v = rows_for(P, 12)
    out = torch.full((12, 4, 128), 7.0, device="cuda", dtype=BF)
    batch = P.batch([2, 9], [5, 0], [20, 0], rows=12)
    gdn.gdn_kv8_append(P.dims, batch, gdn.make_head_norm(eps=1e-6), None, q, k, v, out,
                       P.cache.codes, P.status)
    gdn.raise_on_status(P.status)
    assert (out[:2] == 7).all() and (out[7:] == 7).all()
    want = normed(q[2:7], None, 1e-6, 0.0)
    assert ((out[2:7].double() - want).abs() <= want.abs() * 2.0 ** -8 * 1.01 + 1e-7).all()


def test_queries_in_place():
    P = Paged(1, 70, 4, 1, 256, 64)
    q, k, v = rows_for(P, 70)
    q2, other = q.contiguous(), torch.empty(70, 4, 256, device="cuda", dtype=BF)
    norm = gdn.make_head_norm(torch.rand(256, device="cuda"), None, eps=1e-6)
    inv = torch.logspace(0, -4, 64, device="cuda")
    rope = gdn.make_rope(128, inv, torch.arange(70, device="cuda", dtype=torch.int32), interleaved=True)
    batch = P.batch([0], [70], [70])
    gdn.gdn_kv8_append(P.dims, batch, norm, rope, q, k, v, other, P.cache.codes, P.status)
    gdn.gdn_kv8_append(P.dims, batch, norm, rope, q2, k, v, q2, P.cache.codes, P.status)
    gdn.raise_on_status(P.status)
    assert torch.equal(q2, other)


def _codes_of_normed_keys(P, k, kw, eps, inv, pos):
    """The keys as stored, and those and the exponents that 64 bits give."""
    T, hkv, d = k.shape
    norm = gdn.make_head_norm(None, kw, eps=eps)
    gdn.gdn_kv8_append(P.dims, P.batch([0], [T], [T]), norm, gdn.make_rope(d, inv, pos), None, k, k,
                       None, P.cache.codes, P.status)
    gdn.raise_on_status(P.status)
    turned = rotated(normed(k, kw, eps, 0.0), d, inv, pos)
    want = Blocks(hkv, d)
    want.append(turned, 0)
    return *P.tokens(0, T, P.cache.k, P.cache.k_exp), turned, want


@pytest.mark.parametrize("size,eps", [(1e25, 1e-6), (3e37, 1e-6), (1e-25, 0.0),
                                      (1e-32, 2.0 ** -100), (1e-22, 2.0 ** -126)])
def test_keys_whose_squares_leave_the_range(size, eps):
    """bf16 has fp32's range, the squares of its ends do not fit it. Of a million keys some ten lie
    next to a middle and are formed again; the others as in test_append_and_read."""
    T, d, hkv = 2048, 128, 4
    P = Paged(1, T, 4, hkv, d, 64, seed=22)
    g = torch.Generator(device="cuda").manual_seed(7)
    k = (torch.randn(T, hkv, d, generator=g, device="cuda") * size).to(BF)
    kw = 1 + 0.3 * torch.randn(d, generator=g, device="cuda")
    inv = (1e4 ** -(torch.arange(d // 2, device="cuda").double() / (d // 2))).float()
    pos = torch.arange(7, T + 7, device="cuda", dtype=torch.int32)
    x, e, turned, want = _codes_of_normed_keys(P, k, kw, eps, inv, pos)
    assert torch.isfinite(turned).all() and torch.isfinite(x).all()
    unit = torch.exp2(e.double()).repeat_interleave(BLOCK, 0)[..., None]
    room = grid_step(turned / unit) / 2 * unit + partners(turned, d, False) * 2.0 ** -18
    assert ((x - turned).abs() <= room * (1 + 1e-9)).all()
    # (the same keys as in the test of those next to a middle)
    larger = turned.abs() >= turned.roll(d // 2, -1).abs()
    same = (e == want.e).repeat_interleave(BLOCK, 0)[..., None]
    counted = same & larger & (want.x.abs() >= 2.0 ** -5 * unit)
    assert counted.sum() > 5 * 10 ** 5 and not ((x != want.x) & counted).any()


@pytest.mark.parametrize("size", [2.0 ** 65, -2.0 ** 126, 2.0 ** -80, 1.0])
def test_large_and_small_keys_on_the_middle_of_two_codes(size):
    """Rows of one value come to the weight itself, 17/16: midway between two codes, to the even
    one."""
    P = Paged(1, 16, 2, 1, 64, 16)
    k = torch.full((16, 1, 64), size, device="cuda", dtype=BF)
    kw = torch.full((64,), 1.0625, device="cuda")
    zero = torch.zeros(16, device="cuda", dtype=torch.int32)
    x, e, _, _ = _codes_of_normed_keys(P, k, kw, 0.0, torch.ones(32, device="cuda"), zero)
    assert (e == -8).all() and (x == (1.0 if size > 0 else -1.0)).all()


def test_keys_on_a_middle_that_turn_a_little():
    """A turn that fp32 rounds away, off the middle between two codes: to its side. Those that do
    not turn go to the even code."""
    P = Paged(1, 16, 2, 1, 64, 16)
    k = torch.zeros(16, 1, 64, device="cuda", dtype=BF)
    # pairs (j, 32 + j): x on a middle, y = 1 or -1; x - y 2^-30 is what is rounded
    k[:, 0, 0:4] = torch.tensor([1.0625, 1.0625, 1.1875, 1.1875], device="cuda")
    k[:, 0, 32:36] = torch.tensor([1.0, -1.0, 1.0, -1.0], device="cuda")
    inv = torch.full((32,), 2.0 ** -30, device="cuda")
    pos = torch.zeros(16, device="cuda", dtype=torch.int32)
    pos[8:] = 1
    gdn.gdn_kv8_append(P.dims, P.batch([0], [16], [16]), None, gdn.make_rope(64, inv, pos), None, k, k,
                       None, P.cache.codes, P.status)
    gdn.raise_on_status(P.status)
    x, _ = P.tokens(0, 16, P.cache.k, P.cache.k_exp)
    assert x[0, 0, :4].tolist() == [1.0, 1.0, 1.25, 1.25] and (x[:8] == x[0]).all()
    assert x[8, 0, :4].tolist() == [1.0, 1.125, 1.125, 1.25] and (x[8:] == x[8]).all()


def test_keys_at_far_positions_next_to_the_middle_of_two_codes():
    """Positions next to 2^31: the turn is formed with all of the position's bits, so the codes are
    those of whole-number arithmetic."""
    T, d, hkv = 16384, 128, 4
    P = Paged(1, T, 4, hkv, d, 64, seed=23)
    g = torch.Generator(device="cuda").manual_seed(8)
    k = torch.randn(T, hkv, d, generator=g, device="cuda").to(BF)
    inv = torch.exp2(-torch.rand(d // 2, generator=g, device="cuda"))
    pos = (2 ** 31 - 1 - torch.randint(0, 10 ** 6, (T,), generator=g, device="cuda")).int()
    gdn.gdn_kv8_append(P.dims, P.batch([0], [T], [T]), None, gdn.make_rope(d, inv, pos), None, k, k,
                       None, P.cache.codes, P.status)
    gdn.raise_on_status(P.status)
    # whole turns out of the product in whole numbers: f = n 2^-24, and 2^120 / (2 pi) (pi by
    # Machin's formula)
    def arctan_of(x, one):
        s = term = one // x
        n, sign = 3, -1
        while term:
            term //= x * x
            s, n, sign = s + sign * (term // n), n + 2, -sign
        return s

    one = 1 << 160
    pi = 4 * (4 * arctan_of(5, one) - arctan_of(239, one))
    turn = (1 << 120) * one // (2 * pi)
    ns = [int(f * 2 ** 24) for f in inv.double().tolist()]
    assert all(n / 2 ** 24 == f for n, f in zip(ns, inv.double().tolist()))
    frac = [[(p * n * turn & (1 << 144) - 1) / (1 << 144) for n in ns] for p in pos.tolist()]
    angle = torch.tensor(frac, dtype=torch.float64, device="cuda")[:, None] * (2 * math.pi)
    c, s = torch.cos(angle), torch.sin(angle)
    a, b = k[..., :d // 2].double(), k[..., d // 2:].double()
    turned = torch.cat((a * c - b * s, b * c + a * s), -1)
    want = Blocks(hkv, d)
    want.append(turned, 0)
    x, e = P.tokens(0, T, P.cache.k, P.cache.k_exp)
    unit = torch.exp2(e.double()).repeat_interleave(BLOCK, 0)[..., None]
    larger = turned.abs() >= turned.roll(d // 2, -1).abs()
    same = (e == want.e).repeat_interleave(BLOCK, 0)[..., None]
    counted = same & larger & (want.x.abs() >= 2.0 ** -5 * unit)
    assert counted.sum() > 10 ** 6 and not ((x != want.x) & counted).any()


@pytest.mark.parametrize("d", [64, 256])
def test_keys_below_the_normal_range_without_eps(d):
    """Their size has no fp32 reciprocal."""
    T = 50
    P = Paged(1, T, 2, 2, d, 64)
    q, k, v = (x.clone() for x in rows_for(P, T, spread=0.0))
    q, k = (q.float() * 1e-39).to(BF), (k.float() * 1e-40).to(BF)
    k[:, 1] = v[:, 1]
    inv = (1e4 ** -(torch.arange(d // 2, device="cuda").double() / (d // 2))).float()
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    out = torch.empty_like(q)
    gdn.gdn_kv8_append(P.dims, P.batch([0], [T], [T]), gdn.make_head_norm(eps=0.0),
                       gdn.make_rope(d, inv, pos), q, k, v, out, P.cache.codes, P.status)
    gdn.raise_on_status(P.status)
    turned = rotated(normed(k, None, 0.0, 0.0), d, inv, pos)
    x, e = P.tokens(0, T, P.cache.k, P.cache.k_exp)
    unit = torch.exp2(e.double()).repeat_interleave(BLOCK, 0)[:T, :, None]
    room = grid_step(turned / unit) / 2 * unit + partners(turned, d, False) * 2.0 ** -18
    assert ((x - turned).abs() <= room * (1 + 1e-9)).all()
    yq = normed(q, None, 0.0, 0.0)
    want = rotated(yq, d, inv, pos)
    assert ((out.double() - want).abs() <= want.abs() * 2.0 ** -8 * (1 + 2.0 ** -10)
            + partners(yq, d, False) * 2.0 ** -18).all()
