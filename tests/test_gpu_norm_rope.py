"""gdn_norm_rope against the formula in 64 bits.

Errors: the output's rounding is at most eps / 2 of it. Before it, in fp32: the sum of D squares
(each lane adds up to 16, or up to 16 units of 2 at D = 1024 with single elements, then five
shuffles: fewer than 64 roundings in a row), halved by the root; root, quotient and two products;
cosine and sine within 2^-23 and the angle within 2^-25 of a turn (2^-22.3 rad), and the turn's
three roundings: less than (32 + 8) 2^-24 + 2^-21 < 2^-18 of |x| + |y| of the pair."""
import pytest
import torch

import gated_deltanet_linear_14_gb300 as gdn
from tests.kv8_util import BF, CODE, F32, HF, normed, partners, rotated

pytestmark = pytest.mark.gpu


def check(got, x, w, eps, offset, rd, inv_freq, pos, axis=None, inter=False):
    y = normed(x, w, eps, offset)
    want = rotated(y, rd, inv_freq, pos, axis, inter)
    half = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).tiny * torch.finfo(got.dtype).eps
    room = want.abs() * half * (1 + 2.0 ** -10) + partners(y, rd, inter) * 2.0 ** -18 + tiny
    bad = ((got.double() - want).abs() > room).sum().item()
    assert bad == 0, (bad, (got.double() - want).abs().max().item())


def made(rows, hq, hkv, d, rd, dtype, axes=1, seed=0, spread=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn(rows, hq + 2 * hkv, d, generator=g, device="cuda")
    qkv *= torch.exp(spread * torch.randn(rows, hq + 2 * hkv, 1, generator=g, device="cuda"))
    qkv = qkv.to(dtype)
    qw, kw = (1 + 0.3 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    inv = (1.0 / 1e4 ** (torch.arange(max(rd // 2, 1), device="cuda").double() / max(rd // 2, 1))).float()
    pos = torch.randint(0, 1 << 20, (axes, rows), generator=g, device="cuda", dtype=torch.int32)
    axis = (torch.arange(max(rd // 2, 1), device="cuda") % axes).int()
    return qkv, qw, kw, inv, pos, axis


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("rows,hq,hkv,d,rd,axes,inter,offset", [
    (1, 4, 2, 128, 128, 1, False, 0.0), (3, 16, 2, 256, 64, 1, False, 1.0),
    (1000, 32, 8, 128, 128, 1, True, 0.0), (17, 3, 1, 72, 72, 3, False, 0.0),
    (130, 16, 16, 80, 40, 3, True, 1.0), (5, 2, 1, 64, 0, 1, False, 0.0),
    (70, 6, 2, 96, 2, 1, False, 0.0), (33, 4, 4, 192, 96, 1, False, 0.0),
    (9, 2, 2, 1024, 1024, 1, False, 0.0), (9, 1, 1, 2, 2, 1, True, 0.0),
    (4097, 5, 1, 34, 30, 2, False, 1.0)])
def test_against_the_formula(dtype, rows, hq, hkv, d, rd, axes, inter, offset):
    qkv, qw, kw, inv, pos, axis = made(rows, hq, hkv, d, rd, dtype, axes, seed=d + rows, spread=1.0)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hkv]
    dims = gdn.make_attn_dims(hq, hkv, d, 16, io=CODE[dtype])
    norm = gdn.make_head_norm(qw, kw, eps=1e-6, offset=offset)
    rope = gdn.make_rope(rd, inv, pos, axis=axis, interleaved=inter)
    q_out, k_out = (torch.full((rows, h, d), 7.0, device="cuda", dtype=dtype) for h in (hq, hkv))
    gdn.gdn_norm_rope(dims, norm, rope, q, q_out, k, k_out)
    check(q_out, q, qw, 1e-6, offset, rd, inv, pos, axis, inter)
    check(k_out, k, kw, 1e-6, offset, rd, inv, pos, axis, inter)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,shift", [(128, 1), (1024, 1), (64, 4)])
def test_rows_at_odd_addresses(dtype, d, shift):
    """Rows that begin `shift` elements past an aligned address, with an odd distance."""
    rows, hq = 37, 3
    qkv, qw, kw, inv, pos, _ = made(rows, hq, 1, d, d, dtype)
    gap = hq * d + shift
    store = torch.zeros(rows * gap + shift, device="cuda", dtype=dtype)
    q = torch.as_strided(store, (rows, hq, d), (gap, d, 1), shift)
    q.copy_(qkv[:, :hq])
    out = torch.as_strided(torch.full_like(store, 7.0), (rows, hq, d), (gap, d, 1), shift)
    dims = gdn.make_attn_dims(hq, 1, d, 16, io=CODE[dtype])
    gdn.gdn_norm_rope(dims, gdn.make_head_norm(qw, kw), gdn.make_rope(d, inv, pos[0]), q, out)
    check(out, q, qw, 1e-6, 0.0, d, inv, pos)
    if shift == 1:
        assert (out.as_strided((rows - 1,), (gap,), gap) == 7.0).all()   # between the rows


@pytest.mark.parametrize("d", [128, 1024])
def test_in_place_without_rotation_or_weights(d):
    qkv, _, _, inv, pos, _ = made(50, 4, 4, d, d, BF)
    x = qkv[:, :4].contiguous()
    want = x.clone()
    dims = gdn.make_attn_dims(4, 4, d, 16)
    gdn.gdn_norm_rope(dims, gdn.make_head_norm(eps=1e-5), None, x, x)
    check(x, want, None, 1e-5, 0.0, 0, inv, pos)
    only_k = want.clone()
    gdn.gdn_norm_rope(dims, gdn.make_head_norm(eps=1e-5), gdn.make_rope(d, inv, pos[0]), None,
                      None, only_k, only_k)
    check(only_k, want, None, 1e-5, 0.0, d, inv, pos)


def test_values_whose_squares_leave_the_range():
    """bf16 has fp32's range: squares of 1e25 and of 1e-25 (without eps) do not fit it."""
    qkv, qw, kw, inv, pos, _ = made(8, 4, 1, 128, 128, BF)
    dims = gdn.make_attn_dims(4, 1, 128, 16)
    for size, eps in ((1e25, 1e-6), (3e37, 1e-6), (1e-25, 0.0), (1e-32, 1e-30)):
        q = (qkv[:, :4].float() * size).to(BF)
        out = torch.empty(8, 4, 128, device="cuda", dtype=BF)
        gdn.gdn_norm_rope(dims, gdn.make_head_norm(qw, eps=eps), gdn.make_rope(128, inv, pos[0]), q, out)
        assert torch.isfinite(out).all()
        check(out, q, qw, eps, 0.0, 128, inv, pos)


def test_zero_infinite_and_nan_rows():
    q = torch.ones(4, 2, 64, device="cuda", dtype=BF)
    q[0] = 0.0
    q[1, 0, 3], q[2, 1, 5] = float("inf"), float("nan")
    dims, out = gdn.make_attn_dims(2, 1, 64, 16), torch.empty_like(q)
    gdn.gdn_norm_rope(dims, gdn.make_head_norm(eps=1e-6), None, q, out)
    assert (out[0] == 0).all() and (out[3] == 1).all()
    assert out[1, 0, 3].isnan() and (out[1, 0, :3] == 0).all() and (out[1, 1] == 1).all()
    assert (out[1, 0, 4:] == 0).all()
    assert out[2, 1].isnan().all() and (out[2, 0] == 1).all()


def test_captured_and_replayed_with_other_rows():
    qkv, qw, kw, inv, pos, _ = made(64, 16, 2, 256, 64, BF)
    q, out = qkv[:, :16], torch.empty(64, 16, 256, device="cuda", dtype=BF)
    dims, norm = gdn.make_attn_dims(16, 2, 256, 16), gdn.make_head_norm(qw, kw, offset=1.0)
    rope = gdn.make_rope(64, inv, pos[0])
    gdn.gdn_norm_rope(dims, norm, rope, q, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_norm_rope(dims, norm, rope, q, out)
    qkv.copy_(qkv.flip(0))
    graph.replay()
    check(out, q, qw, 1e-6, 1.0, 64, inv, pos)


@pytest.mark.parametrize("dtype,d,size", [(BF, 128, 1e-39), (BF, 1024, 1e-40), (F32, 128, 1e-39),
                                          (F32, 64, 1e-43), (F32, 1024, 1e-41), (HF, 128, 1e-7)])
def test_rows_below_the_normal_range_without_eps(dtype, d, size):
    """Their size has no fp32 reciprocal."""
    qkv, qw, kw, inv, pos, _ = made(8, 4, 1, d, d, F32)
    dims = gdn.make_attn_dims(4, 1, d, 16, io=CODE[dtype])
    q = (qkv[:, :4] * size).to(dtype)
    q[:, 1] = (qkv[:, 1]).to(dtype)   # (a row of ordinary size beside them)
    out = torch.empty(8, 4, d, device="cuda", dtype=dtype)
    gdn.gdn_norm_rope(dims, gdn.make_head_norm(qw, eps=0.0), gdn.make_rope(d, inv, pos[0]), q, out)
    assert torch.isfinite(out).all()
    check(out, q, qw, 0.0, 0.0, d, inv, pos)
