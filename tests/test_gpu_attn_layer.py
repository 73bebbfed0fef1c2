"""The attention-layer calls (gdn_rope, gdn_kv_append, gdn_attn_plan, gdn_attn)
against plain forms in 64 bits, at sizes and masks where they can go wrong.

Tolerances, from the formats (u = 2^-8 for bf16, 2^-11 for fp16, 2^-24 for
fp32: half a unit in the last place, relative; 8, 11 and 24 significant bits):
  rotation   one rounding of an fp32 value whose own error is a few 2^-24 of
             the pair's length r: |x' - ref| <= u |ref| + 2^-21 r (two
             products, a sum, and cos and sin to a few 2^-24);
  attention  p_j is rounded once to the io type, o once more: |o - ref| <=
             u (sum_j p_j |v_j| / sum_j p_j) + u |o| + 2^-16 max_j |v_j|, the
             last term for fp32 scores (|s| < 16: 2^-24 * 16 * a few) and sums;
             lse: fp32 sums of scores of that size, 2^-16 absolute.
"""
import math

import numpy as np
import pytest
import torch

import gated_deltanet_linear_14_gb300 as gdn

pytestmark = pytest.mark.gpu

CODE = {torch.float32: gdn.GDN_F32, torch.bfloat16: gdn.GDN_BF16, torch.float16: gdn.GDN_F16}
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def i32(v):
    return torch.as_tensor(np.asarray(v, np.int32)).cuda()


def rotate64(x, pos, axis, inv_freq, rd, interleaved, inverse):
    """(rotated, length of each element's pair) in 64 bits."""
    a = pos.double()[axis.long()].t() * inv_freq.double()
    a = -a if inverse else a
    c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
    y, r = x.double().clone(), x.double().abs()
    e = torch.arange(rd // 2, device="cuda")
    i, j = (2 * e, 2 * e + 1) if interleaved else (e, e + rd // 2)
    p, q = x.double()[..., i], x.double()[..., j]
    y[..., i], y[..., j] = p * c - q * s, q * c + p * s
    r[..., i] = r[..., j] = torch.hypot(p, q)
    return y, r


def check_rotated(got, ref, r):
    u = U[got.dtype]
    tiny = 2.0 ** -24 if got.dtype == HF else 0.0  # fp16 subnormals
    bad = (got.double() - ref).abs() > u * ref.abs() + 2.0 ** -21 * r + tiny
    assert not bool(bad.any()), (got.double() - ref).abs().max().item()


def rope_inputs(rows, D, rd, axes, seed, far):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    pos = torch.randint(0, far, (axes, rows), generator=g, device="cuda", dtype=torch.int32)
    freq = (1.0 / 1e6 ** (torch.arange(rd // 2, device="cuda", dtype=torch.float64)
                          / max(rd // 2, 1))).float()
    axis = i32(np.arange(rd // 2) % axes)
    return g, pos, freq, axis


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dt", [BF, HF, F32])
@pytest.mark.parametrize("rows,Hq,Hk,D,rd,axes", [
    (1, 4, 1, 128, 128, 1), (7, 16, 2, 256, 64, 3), (33, 3, 3, 72, 72, 3), (130, 5, 1, 80, 40, 1),
    (65, 2, 2, 64, 2, 1), (3, 1, 1, 1024, 1024, 3), (5, 2, 1, 6, 4, 1), (9, 2, 1, 64, 0, 1)])
def test_rope(rows, Hq, Hk, D, rd, axes, dt, interleaved, inverse):
    g, pos, freq, axis = rope_inputs(rows, D, rd, axes, rows, 1 << 20)
    q = torch.randn(rows, Hq, D, generator=g, device="cuda").to(dt)
    k = torch.randn(rows, Hk, D, generator=g, device="cuda").to(dt)
    qo, ko = torch.full_like(q, 9.0), torch.full_like(k, 9.0)
    dims = gdn.make_attn_dims(Hq, Hk, D, 16, io=CODE[dt])
    rope = gdn.make_rope(rd, freq, pos, axis=axis, interleaved=interleaved)
    gdn.gdn_rope(dims, rope, q, qo, k, ko, inverse=inverse)
    for x, y in ((q, qo), (k, ko)):
        check_rotated(y, *rotate64(x, pos, axis, freq, rd, interleaved, inverse))
        assert torch.equal(y[..., rd:], x[..., rd:])  # what is not rotated passes bit for bit
    # in place, q alone and k alone give the same bits
    qi, ki = q.clone(), k.clone()
    gdn.gdn_rope(dims, rope, qi, qi, inverse=inverse)
    gdn.gdn_rope(dims, rope, None, None, ki, ki, inverse=inverse)
    assert torch.equal(qi, qo) and torch.equal(ki, ko)


@pytest.mark.parametrize("dt,offset,pad", [(BF, 0, 8), (BF, 4, 4), (BF, 1, 3), (F32, 1, 2),
                                           (HF, 2, 5), (F32, 4, 0)])
def test_rope_strides_and_alignment(dt, offset, pad):
    rows, H, D, rd = 11, 3, 64, 32
    g, pos, freq, axis = rope_inputs(rows, D, rd, 1, 5, 4096)
    buf = torch.randn(offset + rows * (H * D + pad), generator=g, device="cuda").to(dt)
    q = buf[offset:].view(rows, H * D + pad)[:, :H * D].view(rows, H, D)
    out = torch.zeros_like(buf)
    qo = out[offset:].view(rows, H * D + pad)[:, :H * D].view(rows, H, D)
    dims = gdn.make_attn_dims(H, H, D, 16, io=CODE[dt])
    gdn.gdn_rope(dims, gdn.make_rope(rd, freq, pos, axis=axis), q, qo)
    check_rotated(qo, *rotate64(q, pos, axis, freq, rd, False, False))
    qo.zero_()
    assert not bool(out.any())  # nothing outside the rows was written


def test_rope_positions_near_and_far():
    """The reduced angle keeps fp32 accuracy at any position that fp32 can hold exactly,
    and for negative ones."""
    pos = i32([[0, 1, -1, -70000, 4095, 4096, 123457, (1 << 24) - 1]])
    freq = torch.tensor([1.0, 0.731, 1e-3, 1e-7], device="cuda")
    axis = i32([0] * 4)
    q = torch.randn(8, 2, 8, device="cuda")
    qo = torch.empty_like(q)
    gdn.gdn_rope(gdn.make_attn_dims(2, 2, 8, 16, io=gdn.GDN_F32), gdn.make_rope(8, freq, pos), q, qo)
    check_rotated(qo, *rotate64(q, pos, axis, freq, 8, False, False))


def test_rope_inverse_is_the_gradient():
    """<rope(x), y> = <x, inverse(y)>, and central differences of a scalar loss."""
    rows, H, D, rd = 4, 2, 16, 12
    g, pos, freq, axis = rope_inputs(rows, D, rd, 3, 8, 500)
    dims = gdn.make_attn_dims(H, H, D, 16, io=gdn.GDN_F32)
    rope = gdn.make_rope(rd, freq, pos, axis=axis, interleaved=True)
    x, w = (torch.randn(rows, H, D, generator=g, device="cuda") for _ in range(2))
    grad = torch.empty_like(w)
    gdn.gdn_rope(dims, rope, w, grad, inverse=True)
    y = torch.empty_like(x)
    gdn.gdn_rope(dims, rope, x, y)
    lhs, rhs = (y.double() * w.double()).sum(), (x.double() * grad.double()).sum()
    assert abs(lhs - rhs) <= 2.0 ** -20 * (x.double().norm() * w.double().norm())
    # the map is linear, so a difference over 2h is exact up to fp32 rounding of y
    for i in ((0, 0, 0), (1, 1, 5), (3, 0, 11), (2, 1, 15)):
        h, hi, lo = 0.5, x.clone(), x.clone()
        hi[i] += h
        lo[i] -= h
        f = []
        for z in (hi, lo):
            o = torch.empty_like(z)
            gdn.gdn_rope(dims, rope, z, o)
            f.append((o.double() * w.double()).sum())
        assert abs((f[0] - f[1]) / (2 * h) - grad[i].double()) <= 2.0 ** -18 * w.double().norm()


# --------------------------------------------------------- cache and attention

class Cache:
    """A step of `rows[r]` new tokens for requests that hold kv[r] tokens after it, groups of
    requests with shared leading pages, in pages dealt at random."""

    def __init__(self, rows, kv, Hq, Hkv, D, ps, dt=BF, groups=(), seed=0, fill="randn",
                 order=None, spare=2):
        rng = np.random.default_rng(seed)
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        self.rows, self.kv = np.asarray(rows), np.asarray(kv)
        self.Hq, self.Hkv, self.D, self.ps, self.dt = Hq, Hkv, D, ps, dt
        R, T = len(rows), int(self.rows.sum())
        self.T = T
        order = np.arange(R) if order is None else np.asarray(order)  # of the rows in the pack
        self.start = np.zeros(R, np.int64)
        self.start[order] = np.cumsum(self.rows[order]) - self.rows[order]
        need = -(-self.kv // ps)
        width = max(int(need.max(initial=0)), 1)
        pool = int(need.sum()) + spare
        deal = rng.permutation(pool)
        self.table = np.full((R, width), -1, np.int64)
        at = 0
        for r in range(R):
            self.table[r, :need[r]] = deal[at:at + need[r]]
            at += need[r]
        for a, n, p in groups:
            self.table[a:a + n, :p] = self.table[a, :p]
        dims_bits = (pool, Hkv, ps, D)
        if fill == "randn":
            self.k, self.v = (torch.randn(dims_bits, generator=self.g, device="cuda").to(dt)
                              for _ in range(2))
        else:  # poison: slots that hold no token are NaN
            self.k, self.v = (torch.full(dims_bits, math.nan, device="cuda", dtype=dt)
                              for _ in range(2))
            for r in range(R):
                for j in range(int(self.kv[r])):
                    p = self.table[r, j // ps]
                    for c in (self.k, self.v):
                        c[p, :, j % ps] = torch.randn(Hkv, D, generator=self.g,
                                                      device="cuda").to(dt)
        self.q = torch.randn(T, Hq, D, generator=self.g, device="cuda").to(dt)
        self.dims = gdn.make_attn_dims(Hq, Hkv, D, ps, io=CODE[dt])
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        gr = [i32([g[i] for g in groups]) for i in range(3)] if groups else []
        self.keep = [i32(self.start), i32(self.rows), i32(self.kv), i32(self.table)] + gr
        self.batch = gdn.make_kv_batch(R, T, int(self.rows.max(initial=0)), pool, *self.keep)

    def plan(self):
        n = gdn.gdn_attn_plan_bytes(self.dims, self.batch)
        self.plan_buf = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        n = gdn.gdn_attn_workspace_bytes(self.dims, self.batch)
        self.ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN words
        gdn.gdn_attn_plan(self.dims, self.batch, self.plan_buf, self.plan_buf.numel(), self.status)

    def attn(self, q=None, lse=True):
        self.plan()
        q = self.q if q is None else q
        o = torch.full((self.T, self.Hq, self.D), 7.0, dtype=self.dt, device="cuda")
        z = torch.full((self.T, self.Hq), 7.0, device="cuda") if lse else None
        gdn.gdn_attn(self.dims, self.batch, self.plan_buf, q, self.k, self.v, o, z, self.ws,
                     self.ws.numel(), self.status)
        return o, z

    def ref(self, r, q=None):
        """(o, bound of |o - ref|, lse) of request r in 64 bits."""
        q = self.q if q is None else q
        n, m, a, G = int(self.kv[r]), int(self.rows[r]), int(self.start[r]), self.Hq // self.Hkv
        pages = torch.as_tensor(self.table[r, :-(-n // self.ps)]).cuda()
        k = self.k[pages].transpose(0, 1).reshape(self.Hkv, -1, self.D)[:, :n].double()
        v = self.v[pages].transpose(0, 1).reshape(self.Hkv, -1, self.D)[:, :n].double()
        x = q[a:a + m].double().reshape(m, self.Hkv, G, self.D)
        s = torch.einsum("mhgd,hnd->mhgn", x, k) / math.sqrt(self.D)
        seen = torch.arange(n, device="cuda") < (torch.arange(m, device="cuda") + n - m + 1)[:, None]
        s = torch.where(seen[:, None, None], s, -math.inf)
        lse = torch.logsumexp(s, -1)
        p = torch.exp(s - lse[..., None])
        v0 = torch.nan_to_num(v)
        o = torch.einsum("mhgn,hnd->mhgd", p, v0)
        u = U[self.dt]
        bound = u * torch.einsum("mhgn,hnd->mhgd", p, v0.abs()) + u * o.abs() + 2.0 ** -16 * v0.abs().max()
        shape = (m, self.Hq, self.D)
        return o.reshape(shape), bound.reshape(shape), lse.reshape(m, self.Hq)

    def check(self, o, z, requests=None, q=None):
        assert int(self.status.item()) == 0
        for r in range(len(self.rows)) if requests is None else requests:
            if self.rows[r] == 0:
                continue
            ref, bound, lse = self.ref(r, q)
            a, m = int(self.start[r]), int(self.rows[r])
            err = (o[a:a + m].double() - ref).abs()
            assert bool((err <= bound).all()), (r, (err / bound).max().item())
            if z is not None:
                e = (z[a:a + m].double() - lse).abs().max().item()
                assert e <= 2.0 ** -16, (r, e)


SHAPES = [(4, 4, 64), (8, 1, 128), (6, 2, 256), (16, 2, 128)]


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("Hq,Hkv,D", SHAPES)
@pytest.mark.parametrize("ps", [16, 64, 256])
def test_attn_decode_lengths(Hq, Hkv, D, ps, dt):
    kv = [1, 2, 15, 16, 17, 63, 127, 128, 129, 255, 256, 257, 1000, 1]
    c = Cache([1] * len(kv), kv, Hq, Hkv, D, ps, dt, seed=1)
    c.check(*c.attn())


@pytest.mark.parametrize("Hq,Hkv,D", SHAPES + [(3, 1, 128), (5, 1, 64), (48, 2, 256), (128, 1, 64)])
def test_attn_rows_of_all_counts(Hq, Hkv, D):
    """Decode, verify and prompt rows in one step, with empty requests between them; the
    rows of the requests lie in another order than the requests."""
    rows = [1, 0, 8, 3, 130, 0, 45, 1, 300, 2]
    kv = [700, 0, 8, 900, 130, 50, 333, 1, 1300, 128]
    c = Cache(rows, kv, Hq, Hkv, D, 32, seed=2, order=[9, 3, 0, 8, 1, 2, 7, 6, 5, 4])
    c.check(*c.attn())


def test_attn_one_long_request():
    """One row over a long cache: the keys are split over the GPU and joined."""
    for rows in (1, 5):
        c = Cache([rows], [40001], 8, 2, 128, 64, seed=3)
        c.check(*c.attn())


@pytest.mark.parametrize("D,G,dt", [(64, 4, BF), (128, 8, HF), (256, 6, BF), (128, 1, BF)])
@pytest.mark.parametrize("ps,pages", [(16, 1), (16, 23), (128, 5)])
def test_attn_shared_prefix(D, G, dt, ps, pages):
    """Two groups, requests outside any group, a prompt inside a group, an empty request."""
    rows = [1, 1, 1, 1, 2, 8, 0, 1, 200, 3]
    base = pages * ps
    kv = [base + 1, base + 70, base + 1, 77, base + 5, base + 8, base, base + 300, base + 200, 40]
    groups = [(0, 3, pages), (4, 5, pages)]
    c = Cache(rows, kv, 2 * G, 2, D, ps, dt, groups=groups, seed=4)
    o, z = c.attn()
    c.check(o, z)


def test_attn_group_reaches_past_a_member():
    """Sharing declared for more pages than a member's rows all see: still right."""
    kv = [64 + 3, 48, 200]
    c = Cache([3, 2, 1], kv, 8, 2, 128, 16, groups=[(0, 3, 3)], seed=5)
    c.check(*c.attn())
    c = Cache([40, 2, 1], [64, 64, 70], 8, 2, 128, 16, groups=[(0, 3, 4)], seed=6)
    c.check(*c.attn())


def test_attn_many_members():
    """A group of more rows than one tile of 128 holds, at every split of its keys."""
    R, pages, ps = 75, 40, 32
    kv = [pages * ps + 1 + 7 * (r % 11) for r in range(R)]
    c = Cache([1 + r % 3 if 7 * (r % 11) > 2 else 1 for r in range(R)], kv, 16, 2, 128, ps,
              groups=[(0, R, pages)], seed=7)
    c.check(*c.attn())


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attn_never_reads_what_holds_no_token(D):
    """NaN in every slot that holds no token, table entries past the length out of range."""
    rows, kv = [1, 3, 1, 40], [1, 37, 130, 161]
    c = Cache(rows, kv, 8, 2, D, 32, seed=8, fill="poison")
    o, z = c.attn()
    c.check(o, z)


def test_attn_infinite_and_nan_keys_stay_with_the_rows_that_see_them():
    """A later row's own key and value may hold NaN or infinity: earlier rows of the same
    request do not see it and stay finite; other requests too."""
    for D, rows, kv, bad in ((128, 9, 140, 135), (64, 150, 300, 200), (256, 4, 4, 2)):
        c = Cache([1, rows, 1], [50, kv, 70], 4, 2, D, 16, seed=9)
        p, j = c.table[1, bad // 16], bad % 16
        c.v[p, :, j, 3] = math.nan
        c.v[p, :, j, 5] = math.inf
        c.k[p, 0, j] = math.inf
        o, z = c.attn()
        c.check(o, z, requests=[0, 2])
        blind = rows - (kv - bad)  # rows that do not see token `bad`
        ref, bound, lse = c.ref(1)
        a = int(c.start[1])
        assert bool(((o[a:a + blind].double() - ref[:blind]).abs() <= bound[:blind]).all())
        assert bool(torch.isnan(o[a + blind:a + rows, :, 3]).all())
        assert not bool(torch.isfinite(o[a + blind:a + rows, :, 5]).any())
        assert bool(torch.isfinite(o[a + blind:a + rows, 2:, 7]).all())


def test_attn_large_scores():
    """Scores far apart: the running maximum moves by more than any threshold, both ways."""
    c = Cache([1, 4], [900, 1500], 4, 2, 128, 32, HF, seed=10)
    c.k.mul_(torch.linspace(0.1, 6.0, c.k.shape[0], device="cuda").half()[:, None, None, None])
    o, z = c.attn()
    for r in range(2):
        ref, bound, lse = c.ref(r)
        a, m = int(c.start[r]), int(c.rows[r])
        # scores up to ~100 here: their fp32 rounding moves p by 2^-24 * 128 * 4, relative
        assert bool(((o[a:a + m].double() - ref).abs() <= bound + 2.0 ** -14).all())
        assert (z[a:a + m].double() - lse).abs().max().item() <= 2.0 ** -14


def test_attn_strided_rows_no_lse_and_repeats():
    c = Cache([1, 8, 33], [400, 900, 33], 8, 2, 128, 64, seed=11)
    wide = torch.randn(c.T, 12, 128, generator=c.g, device="cuda").to(BF)
    q = wide[:, 2:10]
    o1, z1 = c.attn(q=q)
    c.check(o1, z1, q=q)
    o2, none = c.attn(q=q, lse=False)
    assert none is None and torch.equal(o1, o2)  # run to run the same bits


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attn_repeats_bit_for_bit_whatever_ran_before(D):
    """Tiles with few rows: what other calls left in shared and tensor memory
    does not reach them, and a request's bits do not change with its neighbours' values."""
    c = Cache([1, 8, 2], [3000, 2000, 700], 16, 2, D, 64, seed=21)
    other = Cache([5, 40], [900, 1500], 16, 2, D, 32, seed=22)
    other.q.mul_(30)
    ref, z = c.attn()
    for _ in range(4):
        other.attn()
        o, y = c.attn()
        assert torch.equal(o, ref) and torch.equal(y, z)
    c.q[1:9].mul_(8)  # request 1's rows; the plan and the others' values stay
    o, _ = c.attn()
    assert torch.equal(o[0], ref[0]) and torch.equal(o[9:], ref[9:])


def test_attn_rows_outside_any_request_are_not_written():
    c = Cache([2, 3], [40, 50], 4, 2, 64, 16, seed=12)
    c.T += 4
    c.q = torch.cat([c.q, c.q[:4]])
    c.batch.num_rows = c.T
    o, z = c.attn()
    c.check(o, z)
    assert bool((o[5:] == 7).all()) and bool((z[5:] == 7).all())


def test_attn_on_another_stream():
    c = Cache([1, 8], [3000, 2000], 16, 2, 128, 64, seed=13)
    c.plan()
    ref, _ = c.attn()
    o = torch.zeros_like(ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())  # after all that the call reads and writes
    with torch.cuda.stream(side):
        gdn.gdn_attn(c.dims, c.batch, c.plan_buf, c.q, c.k, c.v, o, None, c.ws, c.ws.numel(),
                     c.status)
    side.synchronize()
    assert torch.equal(o, ref)


def test_attn_refuses_a_plan_for_something_else():
    """A plan that was never written, or for other dims or counts: reported, nothing written."""
    c = Cache([1, 4], [100, 90], 8, 2, 128, 16, seed=25)
    good, z = c.attn()

    def run(dims, batch, plan, q):
        o = torch.full_like(q, 7.0)
        ws = torch.empty(gdn.gdn_attn_workspace_bytes(dims, batch), dtype=torch.uint8,
                         device="cuda")
        gdn.gdn_attn(dims, batch, plan, q, c.k, c.v, o, None, ws, ws.numel(), c.status)
        code = int(c.status.item())
        c.status.zero_()
        return code, o

    bad = gdn.CODES["GDN_DEV_STALE_STEP"]
    for fill in (0, 255, 17):
        code, o = run(c.dims, c.batch, torch.full_like(c.plan_buf, fill), c.q)
        assert code == bad and bool((o == 7).all())
    code, o = run(gdn.make_attn_dims(4, 2, 128, 16), c.batch, c.plan_buf, c.q[:, :4].contiguous())
    assert code == bad and bool((o == 7).all())
    one = gdn.make_kv_batch(1, c.T, 4, c.batch.num_pages, *c.keep)
    code, o = run(c.dims, one, c.plan_buf, c.q)
    assert code == bad and bool((o == 7).all())
    code, o = run(c.dims, c.batch, c.plan_buf, c.q)
    assert code == 0 and torch.equal(o, good)


def test_attn_bad_requests_are_skipped():
    rows, kv = [1, 4, 1, 2], [100, 90, 33, 60]
    c = Cache(rows, kv, 8, 2, 128, 16, seed=14)
    c.keep[2][1] = 3  # kv_len below row_len
    o, z = c.attn()
    assert int(c.status.item()) == gdn.CODES["GDN_DEV_BAD_ROWS"]
    c.status.zero_()
    c.check(o, z, requests=[0, 2, 3])
    assert bool((o[1:5] == 7).all())
    c = Cache(rows, kv, 8, 2, 128, 16, seed=15)
    c.keep[3][3, 0] = c.batch.num_pages  # a page past the cache
    o, z = c.attn()
    assert int(c.status.item()) == gdn.CODES["GDN_DEV_BAD_PAGE"]
    c.status.zero_()
    c.check(o, z, requests=[0, 1, 2])


def test_attn_refuses_lengths_that_end_past_32_bits():
    """A tile of keys past the last token must not wrap around: such a request is skipped."""
    c = Cache([1, 1], [200, 64], 1, 1, 64, 256, seed=26)
    width = (1 << 31) // 256
    table = torch.zeros(2, width, dtype=torch.int32, device="cuda")
    table[1, 0] = int(c.table[1, 0])
    c.keep[3] = table
    c.keep[2][0] = (1 << 31) - 200
    c.batch = gdn.make_kv_batch(2, 2, 1, c.batch.num_pages, *c.keep)
    o, z = c.attn()
    assert int(c.status.item()) == gdn.CODES["GDN_DEV_BAD_ROWS"]
    c.status.zero_()
    c.check(o, z, requests=[1])
    assert bool((o[0] == 7).all())
    k0 = c.k.clone()
    k = torch.zeros(2, 1, 64, device="cuda", dtype=BF)
    gdn.gdn_kv_append(c.dims, c.batch, None, None, k, k, None, c.k, c.v, c.status)
    assert int(c.status.item()) == gdn.CODES["GDN_DEV_BAD_ROWS"]
    k0[int(c.table[1, 0]), :, 63] = 0
    assert torch.equal(c.k, k0)


@pytest.mark.parametrize("second", [20, 33])
def test_attn_reports_a_request_of_two_groups(second):
    c = Cache([1] * 64, [2600] * 64, 16, 8, 128, 64, seed=27, groups=[(0, 64, 40)])
    c.check(*c.attn())
    gr = [i32(v) for v in ([0, 31], [32, second], [40, 40])]
    c.batch = gdn.make_kv_batch(64, 64, 1, c.batch.num_pages, *c.keep[:4], *gr)
    c.plan()
    assert int(c.status.item()) == gdn.CODES["GDN_DEV_BAD_ROWS"]


@pytest.mark.parametrize("Hq,Hkv,D,ps,rd,axes,dt,interleaved", [
    (8, 2, 128, 16, 128, 1, BF, False), (16, 2, 256, 64, 64, 3, BF, False),
    (4, 4, 64, 256, 32, 1, HF, True), (3, 1, 64, 32, 6, 3, HF, False)])
def test_append(Hq, Hkv, D, ps, rd, axes, dt, interleaved):
    rows, kv = [1, 0, 8, 37, 1], [1, 20, 40, 37, 513]
    c = Cache(rows, kv, Hq, Hkv, D, ps, dt, seed=16, order=[3, 0, 4, 1, 2])
    qkv = torch.randn(c.T, Hq + 2 * Hkv, D, generator=c.g, device="cuda").to(dt)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    _, pos, freq, axis = rope_inputs(c.T, D, rd, axes, 17, 1 << 18)
    rope = gdn.make_rope(rd, freq, pos, axis=axis, interleaved=interleaved)
    k0, v0 = c.k.clone(), c.v.clone()
    qo = torch.zeros(c.T, Hq, D, dtype=dt, device="cuda")
    gdn.gdn_kv_append(c.dims, c.batch, rope, q, k, v, qo, c.k, c.v, c.status)
    assert int(c.status.item()) == 0
    check_rotated(qo, *rotate64(q, pos, axis, freq, rd, interleaved, False))
    kr, r = rotate64(k, pos, axis, freq, rd, interleaved, False)
    for i in range(len(rows)):
        for t in range(rows[i]):
            j, row = kv[i] - rows[i] + t, int(c.start[i]) + t
            page = int(c.table[i, j // ps])
            check_rotated(c.k[page, :, j % ps], kr[row], r[row])
            assert torch.equal(c.v[page, :, j % ps], v[row])
            k0[page, :, j % ps] = c.k[page, :, j % ps]
            v0[page, :, j % ps] = v[row]
    assert torch.equal(c.k, k0) and torch.equal(c.v, v0)  # nothing else was touched
    # without q, and without a rotation
    k1 = c.k.clone()
    gdn.gdn_kv_append(c.dims, c.batch, rope, None, k, v, None, c.k, c.v, c.status)
    assert torch.equal(c.k, k1)
    gdn.gdn_kv_append(c.dims, c.batch, None, None, k, v, None, c.k, c.v, c.status)
    page = int(c.table[0, 0])
    assert torch.equal(c.k[page, :, 0], k[int(c.start[0])])


def test_append_unaligned_rows():
    c = Cache([3, 2], [20, 2], 2, 1, 64, 16, seed=18)
    buf = torch.randn(1 + 5 * 257, generator=c.g, device="cuda").to(BF)
    row = buf[1:].view(5, 257)
    k, v = row[:, :64].view(5, 1, 64), row[:, 64:128].view(5, 1, 64)
    gdn.gdn_kv_append(c.dims, c.batch, None, None, k, v, None, c.k, c.v, c.status)
    assert torch.equal(c.k[int(c.table[0, 1]), :, 3], k[2]) and torch.equal(
        c.v[int(c.table[1, 0]), :, 1], v[4])


def test_append_bad_requests_are_skipped():
    c = Cache([2, 2, 1], [20, 18, 5], 2, 1, 64, 16, seed=19)
    k, v = (torch.randn(5, 1, 64, generator=c.g, device="cuda").to(BF) for _ in range(2))
    c.keep[3][1, 1] = -1           # the page of request 1's tokens 16 and 17
    k0 = c.k.clone()
    gdn.gdn_kv_append(c.dims, c.batch, None, None, k, v, None, c.k, c.v, c.status)
    assert int(c.status.item()) == gdn.CODES["GDN_DEV_BAD_PAGE"]
    c.status.zero_()
    c.keep[2][0] = 1               # kv_len below row_len
    c.k.copy_(k0)
    gdn.gdn_kv_append(c.dims, c.batch, None, None, k, v, None, c.k, c.v, c.status)
    assert int(c.status.item()) in (gdn.CODES["GDN_DEV_BAD_PAGE"], gdn.CODES["GDN_DEV_BAD_ROWS"])
    k0[int(c.table[2, 0]), :, 4] = k[4]
    assert torch.equal(c.k, k0)


def test_cache_past_32_bits():
    """A cache of more than 2^32 bytes and 2^31 elements: the last page is written and read."""
    Hkv, ps, D, pool = 8, 256, 128, (1 << 31) // (8 * 256 * 128) + 3
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 20 GB")
    c = Cache([1, 1], [300, 10], Hkv, Hkv, D, ps, seed=20)
    c.k = torch.zeros(pool, Hkv, ps, D, dtype=BF, device="cuda")
    c.v = torch.zeros(pool, Hkv, ps, D, dtype=BF, device="cuda")
    c.table = np.array([[3, pool - 1], [pool - 2, -1]])
    c.keep[3].copy_(i32(c.table))
    c.batch.num_pages = pool
    for p in (3, pool - 1, pool - 2):
        c.k[p] = torch.randn(Hkv, ps, D, generator=c.g, device="cuda").to(BF)
        c.v[p] = torch.randn(Hkv, ps, D, generator=c.g, device="cuda").to(BF)
    k, v = (torch.randn(2, Hkv, D, generator=c.g, device="cuda").to(BF) for _ in range(2))
    gdn.gdn_kv_append(c.dims, c.batch, None, None, k, v, None, c.k, c.v, c.status)
    assert torch.equal(c.k[pool - 1, :, 299 - 256], k[0])
    c.check(*c.attn())


def test_step_replayed_from_a_graph():
    """Plan, append and attention captured once: replays read the lengths, rows and cache as
    they are then, and give the bits of plain calls."""
    c = Cache([1, 8, 1, 2], [300, 60, 700, 90], 8, 2, 128, 64, seed=23,
              groups=[(0, 4, 0)])
    k, v = (torch.randn(c.T, 2, 128, generator=c.g, device="cuda").to(BF) for _ in range(2))
    q_rot, o = torch.empty_like(c.q), torch.empty_like(c.q)
    _, pos, freq, axis = rope_inputs(c.T, 128, 64, 1, 24, 1 << 16)
    rope = gdn.make_rope(64, freq, pos, axis=axis)
    c.plan()

    def step():
        gdn.gdn_attn_plan(c.dims, c.batch, c.plan_buf, c.plan_buf.numel(), c.status)
        gdn.gdn_kv_append(c.dims, c.batch, rope, c.q, k, v, q_rot, c.k, c.v, c.status)
        gdn.gdn_attn(c.dims, c.batch, c.plan_buf, q_rot, c.k, c.v, o, None, c.ws, c.ws.numel(),
                     c.status)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for shift in (0, 3, 20):  # every request goes on: within its pages
        c.keep[2].copy_(i32(np.minimum(c.kv + shift, -(-c.kv // 64) * 64)))
        c.q.add_(0.25)
        o.zero_()
        graph.replay()
        got = o.clone()
        step()
        assert torch.equal(got, o) and int(c.status.item()) == 0 and bool(o.any())
