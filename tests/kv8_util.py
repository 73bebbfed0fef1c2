"""64-bit forms of the norms of queries and keys and of the 8-bit cache, and steps for its tests."""
import torch

import gated_deltanet_linear_14_gb300 as gdn
from gated_deltanet_linear_14_gb300.pages import Kv8Cache, torch_dtype

BLOCK, TOP, RANGE = 16, 448.0, 60
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
CODE = {BF: gdn.GDN_BF16, HF: gdn.GDN_F16, F32: gdn.GDN_F32}


def i32(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def normed(x, w, eps, offset):
    """Rows [t][heads][d] in 64 bits, normed head by head (w None: no weight)."""
    y = x.double()
    y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps)
    return y if w is None else y * (offset + w.double())


def rotated(y, rd, inv_freq, positions, axis=None, interleaved=False):
    """Rows in 64 bits with the pairs of the first rd elements turned; positions [axes][rows]."""
    if rd == 0:
        return y
    positions = positions.view(-1, positions.shape[-1]).double()
    ax = torch.zeros(rd // 2, dtype=torch.long, device=y.device) if axis is None else axis.long()
    angle = (positions[ax].t() * inv_freq.double())[:, None]
    c, s = torch.cos(angle), torch.sin(angle)
    z = y.clone()
    a, b = ((slice(0, rd, 2), slice(1, rd, 2)) if interleaved
            else (slice(0, rd // 2), slice(rd // 2, rd)))
    z[..., a] = y[..., a] * c - y[..., b] * s
    z[..., b] = y[..., b] * c + y[..., a] * s
    return z


def partners(y, rd, interleaved):
    """|x| + |y| of each element's pair (the element alone where it does not turn): what rounding
    errors of a turned value are relative to."""
    s = y.abs().clone()
    a, b = ((slice(0, rd, 2), slice(1, rd, 2)) if interleaved
            else (slice(0, rd // 2), slice(rd // 2, rd)))
    both = y[..., a].abs() + y[..., b].abs()
    s[..., a], s[..., b] = both, both
    return s


def least_exponent(top):
    e = torch.arange(-RANGE, RANGE + 1, device=top.device)
    fits = top[..., None] <= TOP * torch.exp2(e.double())
    return torch.where(fits.any(-1), fits.int().argmax(-1) - RANGE, RANGE)


def grid_step(z):
    """The distance of e4m3 values around z."""
    return torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)


def on_grid(x, e):
    unit = torch.exp2(e.double())
    z = x / unit
    s = grid_step(z)
    y = torch.clamp(torch.round(z / s) * s, -TOP, TOP) * unit
    return torch.where(torch.isfinite(x), y, torch.nan)


class Blocks:
    """One request's history of one head kind: values as stored, 64 bits, [tokens][heads][d], and
    exponents [blocks][heads], appended to as the calls are."""

    def __init__(self, heads, d):
        self.x = torch.zeros(0, heads, d, dtype=torch.float64, device="cuda")
        self.e = torch.zeros(0, heads, dtype=torch.long, device="cuda")

    def append(self, x, at):
        """Rows x become tokens at, at + 1, ...: those from there on are replaced."""
        self.x, b = self.x[:at], at // BLOCK
        e_old = self.e[b] if at % BLOCK else None
        self.e = self.e[:b]
        done = 0
        while done < len(x):
            n = min(BLOCK - (at + done) % BLOCK, len(x) - done)
            part = x[done:done + n]
            fine = torch.where(torch.isfinite(part), part.abs(), 0.0)
            e = least_exponent(fine.amax(-1).amax(0))
            old = self.x[b * BLOCK:]
            if e_old is not None:
                e, e_old = torch.maximum(e, e_old), None
                old = on_grid(old, e[None, :, None])
            self.x = torch.cat((self.x[:b * BLOCK], old, on_grid(part, e[None, :, None])))
            self.e = torch.cat((self.e, e[None]))
            done, b = done + n, b + 1


class Paged:
    """An 8-bit cache with a page table of shuffled pages for `tokens` tokens a request."""

    def __init__(self, requests, tokens, hq=4, hkv=2, d=128, ps=16, dtype=BF, seed=0, spare=3):
        self.dims = gdn.make_attn_dims(hq, hkv, d, ps, io=CODE[dtype])
        self.width = -(-tokens // ps)
        g = torch.Generator().manual_seed(seed)
        order = torch.randperm(requests * self.width + spare, generator=g)[:requests * self.width]
        self.table = order.view(requests, self.width).int().cuda()
        self.cache = Kv8Cache(self.dims, requests * self.width + spare)
        for c, e in ((self.cache.k, self.cache.k_exp), (self.cache.v, self.cache.v_exp)):
            c.view(torch.uint8).fill_(0x7F)   # NaN wherever nothing is written
            e.fill_(99)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def batch(self, row_start, row_len, kv_len, rows=None, max_rows=None, groups=()):
        rows = sum(row_len) if rows is None else rows
        return gdn.make_kv_batch(len(row_len), rows, max(row_len) if max_rows is None else max_rows,
                                 self.cache.num_pages, i32(row_start), i32(row_len), i32(kv_len),
                                 self.table, *groups)

    def tokens(self, r, n, codes, exps):
        """Tokens 0 .. n - 1 of request r in 64 bits [n][heads][d], and exponents [blocks][heads]."""
        ps = self.dims.page_size
        pages = self.table[r, :-(-n // ps)].long()
        x = Kv8Cache.values(codes.view(torch.uint8)[pages].view(codes.dtype), exps[pages])
        x = x.double().transpose(1, 2).reshape(-1, *codes.shape[1:2], codes.shape[3])[:n]
        e = exps[pages].long().transpose(1, 2).reshape(-1, codes.shape[1])[:-(-n // BLOCK)]
        return x, e


__all__ = [n for n in dir() if not n.startswith("_")]
assert torch_dtype(gdn.GDN_BF16) is BF
