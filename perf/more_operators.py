"""What is measured of the attention layers' 8-bit cache and of their query and key norms.

Four operators, for the softmax-attention layers that a hybrid stack puts
between its Gated DeltaNet layers:

  norm    RMS norm of query and key rows for each head, and the rotary
          positions in the same pass;
  append  keys normed and rotated, and values, written to a paged cache as
          8-bit floating-point codes (e4m3) with a power of two as the scale
          of each block of 16 tokens and head; the queries normed and rotated
          on the way; then what the step touched of the cache, read back;
  read    a cache's tokens back as rows of 16 bits;
  attn    causal attention of a step's query rows over the 8-bit cache, for
          requests of which groups may share leading pages.

``run`` computes the plain form in 32 bits (angles and values that are about to
be rounded to 8 bits in 64) with elementary torch operations, or, where ``own``
is true, calls the framework's entry points. ``exact`` is the definition in 64
bits, request by request.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
BLOCK = 16          # tokens of a block with one scale
TOP = 448.0         # the largest e4m3 value
RANGE = 60          # scales lie between 2^-60 and 2^60
EPS = 1.0e-6


# ------------------------------------------------------------------- cases

def _case(op, name, **kw):
    c = {"name": name, "op": op, "dtype": "bf16", "hq": 32, "hkv": 8, "d": 128, "rd": 128,
         "axes": 1, "interleaved": False, "requests": 1, "rows_min": 1, "rows_max": 1,
         "kv_min": 0, "kv_max": 0, "page": 64, "groups": 0, "shared": 0, "base": 1.0e6,
         "first": 0, "short": 0, "offset": 0.0, "mix": 1}
    c.update(kw)
    return c


def listed():
    return [
        # a decode step's rows of 64 requests, rotary on a quarter of wide heads, weights around 0
        _case("norm", "norm_decode", requests=64, hq=16, hkv=2, d=256, rd=64, first=120000,
              offset=1.0),
        # prompts of ragged lengths whose keys go to a 16-bit cache
        _case("norm", "norm_prompt", requests=8, rows_min=1000, rows_max=4096),
        # the smallest step: one request, one new token inside a block
        _case("append", "append8_one", kv_min=776, kv_max=776),
        # speculative candidates and short prompts packed into one step, three axes, wide heads
        _case("append", "append8_mixed", requests=40, rows_min=8, rows_max=400, kv_max=4000,
              hq=16, hkv=2, d=256, rd=64, axes=3, page=16, short=80, offset=1.0),
        # long prompts enter the cache at once
        _case("append", "append8_prompt", requests=4, rows_min=8192, rows_max=8192, dtype="f16",
              page=128),
        # the last few tokens of many requests, e.g. for a draft head that attends to them
        _case("read", "read8_tail", requests=64, rows_min=1, rows_max=40, kv_max=4000, page=16),
        # whole documents back to 16 bits, to hand them to another machine or another layout
        _case("read", "read8_long", requests=6, rows_min=12000, rows_max=32768, kv_max=0),
        # the smallest attention call: one token of one request, a few hundred keys
        _case("attn", "attn8_one", kv_min=512, kv_max=512),
        # a decode batch of ragged lengths with nothing shared
        _case("attn", "attn8_decode", requests=64, kv_max=32767, page=16),
        # a decode batch of wide heads, eight queries to a key head
        _case("attn", "attn8_wide", requests=96, hq=16, hkv=2, d=256, rd=64, kv_min=2000,
              kv_max=12000),
        # speculative verification (1 + 7 rows) in four groups, each behind its own prefix
        _case("attn", "attn8_verify", requests=64, rows_min=8, rows_max=8, dtype="f16",
              kv_max=900, groups=4, shared=4096, page=32),
        # prompt pieces over a shared document: long on both sides, so compute counts
        _case("attn", "attn8_prompt", requests=4, rows_min=1500, rows_max=2048, kv_max=512,
              groups=1, shared=8192),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 280.0)


def draw(rng):
    """One more case of the same ranges; never dearer than the dearest listed one."""
    most = max(_cost(c) for c in listed() if c["op"] == "attn")
    while True:
        op = rng.choice(["norm", "append", "read", "attn", "attn", "attn"])
        hkv = rng.choice([1, 2, 4, 8])
        g = rng.choice([1, 2, 3, 4, 6, 8, 16])
        c = _case(op, "drawn", hkv=hkv, hq=hkv * g, dtype=rng.choice(["bf16", "bf16", "f16"]),
                  page=rng.choice([16, 32, 64, 128]), mix=rng.randrange(1 << 20))
        if c["hq"] > 64:
            continue
        c["offset"] = rng.choice([0.0, 1.0])
        if op == "norm":
            c["d"] = rng.choice([64, 72, 80, 96, 128, 192, 256])
            c["rd"] = rng.choice([c["d"], c["d"], c["d"] // 2])
            c["dtype"] = rng.choice(["bf16", "f16", "f32"])
            c["requests"] = _log(rng, 1, 64)
            if rng.random() < 0.7:
                c["rows_max"] = _log(rng, 1, 16384 // c["requests"])
                c["rows_min"] = max(1, c["rows_max"] // 3)
        else:
            c["d"] = rng.choice([64, 128, 256])
            c["rd"] = rng.choice([c["d"], 64])
            c["requests"] = _log(rng, 1, 128)
            kind = rng.random()
            if kind < 0.35:
                c["rows_min"] = c["rows_max"] = 1
            elif kind < 0.6:
                c["rows_min"], c["rows_max"] = 1, rng.randint(2, 8)
            else:
                c["rows_max"] = _log(rng, 9, 2048 if op == "attn" else 16384)
                c["rows_min"] = rng.randint(1, c["rows_max"])
            c["kv_max"] = _log(rng, 1, 24000)
            c["kv_min"] = rng.randint(0, c["kv_max"])
            if op == "attn" and rng.random() < 0.5:
                c["groups"] = rng.randint(1, max(1, min(4, c["requests"])))
                c["shared"] = _log(rng, 64, 32768)
        c["axes"] = rng.choice([1, 1, 3])
        c["interleaved"] = rng.random() < 0.3
        c["base"] = rng.choice([1.0e4, 1.0e6])
        c["first"] = rng.choice([0, _log(rng, 1, 200000)])
        t, r = int(_lengths(c)[0].sum()), c["requests"]
        kv = int(_lengths(c)[1].max())
        # the plain form pads rows and keys: what it holds stays within the card
        pad = r * c["rows_max"] * c["hq"] * kv * 4.0 * 3 + r * kv * c["hkv"] * c["d"] * 4.0 * 4
        if t <= (200000 if op == "read" else 40000) and _cost(c) <= most and (
                op != "attn" or pad < 4.0e10):
            del c["name"]
            return c


def _lengths(case):
    """(new rows, keys after the step) of each request, from the case alone: the first
    `short` percent have rows_min rows; kv_min to kv_max own keys stand before the rows."""
    rng = np.random.default_rng(case["mix"])
    n = case["requests"]
    rows = rng.integers(case["rows_min"], case["rows_max"] + 1, n)
    before = rng.integers(case["kv_min"], case["kv_max"] + 1, n)
    rows[: n * case["short"] // 100] = case["rows_min"]
    before = before + _shared_pages(case) * case["page"]
    return rows.astype(np.int64), (before + rows).astype(np.int64)


def _shared_pages(case):
    return case["shared"] // case["page"] if case["groups"] else 0


def _groups(case):
    """(first request, requests) of each group of consecutive requests."""
    edges = np.linspace(0, case["requests"], case["groups"] + 1).astype(np.int64)
    return edges[:-1], np.diff(edges)


def _tail(rows, kv):
    """Rows that an append touches: its own, and the older tokens of their first block."""
    return rows + (kv - rows) % BLOCK


def work(case):
    e, d, hq, hkv = SIZE[case["dtype"]], case["d"], case["hq"], case["hkv"]
    rows, kv = _lengths(case)
    t = int(rows.sum())
    # squares, their scale and weight for every element; six operations a rotated pair of values
    norm = 4.0 * t * (hq + hkv) * d + 3.0 * t * (hq + hkv) * case["rd"]
    if case["op"] == "norm":
        return {"bytes": 2.0 * t * (hq + hkv) * d * e + 4.0 * t * case["axes"], "flops": norm}
    code = 1.0 + 1.0 / (BLOCK * d)  # of an element in the cache, its share of a scale with it
    if case["op"] == "append":
        back = float(_tail(rows, kv).sum())
        return {"bytes": 2.0 * t * hq * d * e + 2.0 * t * hkv * d * (e + code)
                + 2.0 * back * hkv * d * (code + e) + 4.0 * t * case["axes"],
                "flops": norm + 4.0 * t * hkv * d}
    if case["op"] == "read":
        return {"bytes": 2.0 * t * hkv * d * (code + e), "flops": 2.0 * t * hkv * d}
    # each key and value once for all that share it; each row in, its output and its lse out
    shared = _shared_pages(case) * case["page"]
    keys = float((kv - shared).sum()) + float(shared * case["groups"])
    pairs = float((rows * kv - rows * (rows - 1) // 2).sum())
    return {"bytes": 2.0 * keys * hkv * d * code + 2.0 * t * hq * d * e + 4.0 * t * hq,
            "flops": 4.0 * pairs * hq * d}


# ------------------------------------------------------------------ inputs

def _positions(case, rows, kv, gen):
    """int32 [axes][rows]: the place of each row in its sequence; on three axes, of a
    video's patches (a frame of 24 x 32), each axis with its own."""
    t = np.concatenate([np.arange(b - a, b) for a, b in zip(rows, kv)])
    t = t + case["first"]
    if case["axes"] == 1:
        p = t[None]
    else:
        p = np.stack([case["first"] + t // 768, (t // 32) % 24 + t // 768, t % 32 + t // 768])
    p = torch.from_numpy(p.astype(np.int32)).cuda()
    # new inputs for each seed: the whole step somewhere else
    return (p + torch.randint(0, 64, (1,), generator=gen, device="cuda", dtype=torch.int32)).contiguous()


def _exponent(top):
    """The least e with top <= 448 2^e, within the range, as int64 (top >= 0, any type)."""
    m, x = torch.frexp(top)
    e = x.long() - torch.where(m <= 0.875, 9, 8)
    return torch.where(top > 0, e, -RANGE).clamp_(-RANGE, RANGE)


def _take(codes, *at):
    return codes.view(torch.uint8)[at].view(codes.dtype)


def _put(codes, at, x):
    codes.view(torch.uint8)[at] = x.to(codes.dtype).view(torch.uint8)


def _quantised(pool, hkv, ps, d, gen):
    """A cache that holds normal values of different size from page to page and head to head:
    codes [pool][hkv][ps][d] and exponents int8 [pool][hkv][ps / 16]."""
    codes = torch.empty(pool, hkv, ps, d, device="cuda", dtype=torch.float8_e4m3fn)
    exps = torch.empty(pool, hkv, ps // BLOCK, device="cuda", dtype=torch.int8)
    step = max(1, (1 << 28) // (hkv * ps * d))
    for a in range(0, pool, step):
        n = min(step, pool - a)
        x = torch.randn(n, hkv, ps // BLOCK, BLOCK * d, generator=gen, device="cuda",
                        dtype=torch.bfloat16)
        x *= torch.exp(0.5 * torch.randn(n, hkv, 1, 1, generator=gen, device="cuda"))
        e = _exponent(x.abs().amax(-1).float())
        exps[a:a + n] = e.to(torch.int8)
        codes[a:a + n] = torch.ldexp(x.float(), -e[..., None]).view(n, hkv, ps, d).to(codes.dtype)
    return codes, exps


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    dt, d, hq, hkv, ps = TYPES[case["dtype"]], case["d"], case["hq"], case["hkv"], case["page"]
    rows, kv = _lengths(case)
    t, n = int(rows.sum()), case["requests"]

    def randn(*shape, dtype=dt):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)

    def i32(v):
        return torch.from_numpy(np.ascontiguousarray(v, dtype=np.int32)).cuda()

    s = {"case": dict(case), "t": t}
    if case["op"] in ("norm", "append"):
        half = case["rd"] // 2
        s["inv_freq"] = (1.0 / case["base"] ** (torch.arange(half, device="cuda", dtype=torch.float64)
                                                / half)).float()
        # time, height and width take turns over the frequencies
        s["axis"] = i32(np.arange(half) % case["axes"])
        s["pos"] = _positions(case, rows, kv, gen)
        # trained weights lie around one
        s["qw"], s["kw"] = (1.0 - case["offset"] + 0.2 * randn(d, dtype=torch.float32)
                            for _ in range(2))
        # the projections write q, k and v of a row side by side
        qkv = randn(t, hq + 2 * hkv, d)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    elif case["op"] == "attn":
        s["q"] = randn(t, hq, d)
    if case["op"] in ("norm", "append"):
        s["q_out"] = torch.empty(t, hq, d, device="cuda", dtype=dt)
    if case["op"] == "norm":
        s["k_out"] = torch.empty(t, hkv, d, device="cuda", dtype=dt)
    else:
        # pages dealt at random from a pool a little larger than what is in use
        shared = _shared_pages(case)
        need = -(-kv // ps)
        width = int(need.max())
        own_pages = need - shared
        pool = int(own_pages.sum()) + shared * case["groups"] + 3
        deal = rng.permutation(pool)
        table = np.zeros((n, width), np.int64)
        at = 0
        if case["groups"]:
            for a, c in zip(*_groups(case)):
                table[a:a + c, :shared] = deal[at:at + shared]
                at += shared
        for r in range(n):
            table[r, shared:need[r]] = deal[at:at + own_pages[r]]
            at += own_pages[r]
        s["table"] = i32(table)
        s["k_cache"], s["k_exp"] = _quantised(pool, hkv, ps, d, gen)
        s["v_cache"], s["v_exp"] = _quantised(pool, hkv, ps, d, gen)
        s["row_start"], s["row_len"], s["kv_len"] = i32(np.cumsum(rows) - rows), i32(rows), i32(kv)
        s["row_req"] = torch.from_numpy(np.repeat(np.arange(n), rows)).cuda()
        s["row_t"] = torch.from_numpy(np.concatenate([np.arange(a) for a in rows])).cuda()
        if case["groups"]:
            a, c = _groups(case)
            s["group"] = (i32(a), i32(c), i32(np.full(case["groups"], shared)))
    if case["op"] in ("append", "read"):
        back = _tail(rows, kv) if case["op"] == "append" else rows
        s["back_start"], s["back_len"] = i32(np.cumsum(back) - back), i32(back)
        s["back_req"] = torch.from_numpy(np.repeat(np.arange(n), back)).cuda()
        s["back_at"] = torch.from_numpy(
            np.concatenate([np.arange(b - a, b) for a, b in zip(back, kv)])).cuda()
        s["back_most"], s["back"] = int(back.max()), int(back.sum())
        s["k_back"], s["v_back"] = (torch.empty(s["back"], hkv, d, device="cuda", dtype=dt)
                                    for _ in range(2))
    if case["op"] == "attn":
        s["o"], s["lse"] = torch.empty_like(s["q"]), torch.empty(t, hq, device="cuda")
    if own:
        _handles(case, s, rows)
    return s


def _handles(case, s, rows):
    """What a user's program keeps: dims, the step's row map, and for attention the plan of
    the step's lengths, which all attention layers of the step share, and its workspace."""
    import gated_deltanet_linear_14_gb300 as gdn
    code = {"bf16": gdn.GDN_BF16, "f16": gdn.GDN_F16, "f32": gdn.GDN_F32}[case["dtype"]]
    s["gdn"] = gdn
    s["dims"] = gdn.make_attn_dims(case["hq"], case["hkv"], case["d"], case["page"], io=code)
    if case["op"] in ("norm", "append"):
        s["norm"] = gdn.make_head_norm(s["qw"], s["kw"], eps=EPS, offset=case["offset"])
        s["rope"] = gdn.make_rope(case["rd"], s["inv_freq"], s["pos"], axis=s["axis"],
                                  interleaved=case["interleaved"])
    if case["op"] == "norm":
        return
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    s["cache"] = gdn.make_kv8_cache(s["k_cache"], s["v_cache"], s["k_exp"], s["v_exp"])
    pages = s["k_cache"].shape[0]
    s["batch"] = gdn.make_kv_batch(case["requests"], s["t"], int(rows.max()), pages,
                                   s["row_start"], s["row_len"], s["kv_len"], s["table"],
                                   *s.get("group", ()))
    if case["op"] != "attn":
        s["back_batch"] = gdn.make_kv_batch(case["requests"], s["back"], s["back_most"], pages,
                                            s["back_start"], s["back_len"], s["kv_len"],
                                            s["table"])
    else:
        nbytes = gdn.gdn_kv8_attn_plan_bytes(s["dims"], s["batch"])
        s["plan"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        nbytes = gdn.gdn_kv8_attn_workspace_bytes(s["dims"], s["batch"])
        s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        gdn.gdn_kv8_attn_plan(s["dims"], s["batch"], s["plan"], s["plan"].numel(), s["status"])


# --------------------------------------------------------------- plain form

def _normed_rotated(s, x, w, to64=False):
    """Rows [t][heads][d] normed per head and rotated; angles, and with `to64` all, in 64 bits."""
    case = s["case"]
    rd = case["rd"]
    y = x.double() if to64 else x.float()
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * (w.to(y.dtype) + case["offset"])
    angle = s["pos"][s["axis"].long()].t().double() * s["inv_freq"].double()
    cos, sin = torch.cos(angle).to(y.dtype)[:, None], torch.sin(angle).to(y.dtype)[:, None]
    r, rest = y[..., :rd], y[..., rd:]
    if case["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r[..., :rd // 2], r[..., rd // 2:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((r, rest), -1)


def _plain_write(s, x, codes, exps):
    """Rows x (64 bits) of the step into the cache, block by block."""
    ps = s["case"]["page"]
    pool, hkv, _, d = codes.shape
    nb = ps // BLOCK
    table, start = s["table"].long(), (s["kv_len"] - s["row_len"]).long()
    at = start[s["row_req"]] + s["row_t"]
    page, slot = table[s["row_req"], at // ps], at % ps
    # the blocks (of all pages, one after the other) and the largest new value in each
    block = page * nb + slot // BLOCK
    top = torch.zeros(pool * nb, hkv, device=x.device, dtype=x.dtype)
    top.scatter_reduce_(0, block[:, None].expand(-1, hkv), x.abs().amax(-1), "amax")
    touched = torch.zeros(pool * nb, device=x.device, dtype=torch.bool)
    touched[block] = True
    # a request's first block may hold older tokens, whose scale only grows
    first = table[torch.arange(len(start), device=x.device), start // ps] * nb + start % ps // BLOCK
    kept = torch.zeros_like(touched)
    kept[first] = start % BLOCK > 0
    before = exps.transpose(1, 2).reshape(pool * nb, hkv).long()
    e = _exponent(top)
    e = torch.where(kept[:, None], torch.maximum(e, before), e)
    e = torch.where(touched[:, None], e, before)
    view = codes.view(pool, hkv, nb, BLOCK, d)
    p, b = first // nb, first % nb
    # (an older code times a power of two is exact in 32 bits)
    there = _take(view, p, slice(None), b).float()
    old = torch.ldexp(there, (before - e)[first][..., None, None])
    keep = torch.arange(BLOCK, device=x.device) < (start % BLOCK)[:, None]
    _put(view, (p, slice(None), b), torch.where(keep[:, None, :, None], old, there))
    _put(codes, (page, slice(None), slot),
         torch.ldexp(x, -e[block][..., None]).float().clamp(-TOP, TOP))
    exps.copy_(e.view(pool, nb, hkv).transpose(1, 2))


def _plain_read(s, codes, exps):
    ps = s["case"]["page"]
    page = s["table"].long()[s["back_req"], s["back_at"] // ps]
    slot = s["back_at"] % ps
    x = torch.ldexp(_take(codes, page, slice(None), slot).float(), exps[page, :, slot // BLOCK][..., None])
    return x.to(TYPES[s["case"]["dtype"]])


def _plain_append(s):
    _plain_write(s, _normed_rotated(s, s["k"], s["kw"], to64=True), s["k_cache"], s["k_exp"])
    _plain_write(s, s["v"].double(), s["v_cache"], s["v_exp"])
    return (_normed_rotated(s, s["q"], s["qw"]).to(s["q"].dtype),
            _plain_read(s, s["k_cache"], s["k_exp"]), _plain_read(s, s["v_cache"], s["v_exp"]))


def _plain_attn(s):
    case = s["case"]
    n, hkv, d, ps = case["requests"], case["hkv"], case["d"], case["page"]
    g, tm = case["hq"] // hkv, case["rows_max"]
    table = s["table"].long()
    width = table.shape[1] * ps

    def rows_of(codes, exps):
        x = _take(codes, table).float().view(n, -1, hkv, ps // BLOCK, BLOCK * d)
        x = torch.ldexp(x, exps[table][..., None])
        return x.view(n, -1, hkv, ps, d).transpose(1, 2).reshape(n, hkv, width, d)

    step = torch.arange(tm, device="cuda")
    row = (s["row_start"].long()[:, None] + step).clamp_(max=s["t"] - 1)
    q = s["q"][row].float().view(n, tm, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, g * tm, d)
    score = torch.matmul(q, rows_of(s["k_cache"], s["k_exp"]).transpose(-1, -2)) * (1.0 / math.sqrt(d))
    last = (s["kv_len"].long() - s["row_len"].long())[:, None] + step  # the row's own key
    seen = torch.arange(width, device="cuda") <= last[..., None]
    score.view(n, hkv, g, tm, width).masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    score = score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    o = torch.matmul(score, rows_of(s["v_cache"], s["v_exp"])) / total
    lse = (top + total.log()).squeeze(-1)
    o = o.view(n, hkv, g, tm, d).permute(0, 3, 1, 2, 4).reshape(n, tm, hkv * g, d)
    lse = lse.view(n, hkv, g, tm).permute(0, 3, 1, 2).reshape(n, tm, hkv * g)
    return o[s["row_req"], s["row_t"]].to(s["q"].dtype), lse[s["row_req"], s["row_t"]]


def run(s):
    op = s["case"]["op"]
    if own:
        gdn = s["gdn"]
        if op == "norm":
            gdn.gdn_norm_rope(s["dims"], s["norm"], s["rope"], s["q"], s["q_out"], s["k"],
                              s["k_out"])
            return s["q_out"], s["k_out"]
        if op == "attn":
            gdn.gdn_kv8_attn(s["dims"], s["batch"], s["plan"], s["q"], s["cache"], s["o"],
                             s["lse"], s["workspace"], s["workspace"].numel(), s["status"])
            return s["o"], s["lse"]
        if op == "append":
            gdn.gdn_kv8_append(s["dims"], s["batch"], s["norm"], s["rope"], s["q"], s["k"],
                               s["v"], s["q_out"], s["cache"], s["status"])
        gdn.gdn_kv8_read(s["dims"], s["back_batch"], s["cache"], s["k_back"], s["v_back"],
                         s["status"])
        back = s["k_back"], s["v_back"]
        return (s["q_out"],) + back if op == "append" else back
    if op == "norm":
        return (_normed_rotated(s, s["q"], s["qw"]).to(s["q"].dtype),
                _normed_rotated(s, s["k"], s["kw"]).to(s["k"].dtype))
    if op == "append":
        return _plain_append(s)
    if op == "read":
        return _plain_read(s, s["k_cache"], s["k_exp"]), _plain_read(s, s["v_cache"], s["v_exp"])
    return _plain_attn(s)


# ------------------------------------------------------------- in 64 bits

def _turned(case, s, x, w):
    """Normed by the mean square, then rotated as complex numbers: pair j of row i times
    e^{i position frequency}."""
    rd = case["rd"]
    y = x.double()
    y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / case["d"] + EPS)
    y = y * (case["offset"] + w.double())
    angle = s["pos"].double()[s["axis"].long()].t() * s["inv_freq"].double()
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    if case["interleaved"]:
        z = torch.view_as_complex(y[..., :rd].reshape(*y.shape[:-1], rd // 2, 2).contiguous()) * turn
        y[..., :rd] = torch.view_as_real(z).reshape(*y.shape[:-1], rd)
    else:
        z = torch.complex(y[..., :rd // 2].contiguous(), y[..., rd // 2:rd].contiguous()) * turn
        y[..., :rd // 2], y[..., rd // 2:rd] = z.real, z.imag
    return y


def _on_grid(x, e):
    """x on the grid of e4m3 values times 2^e, ties to even, as float64."""
    unit = torch.exp2(e.double())
    z = x / unit
    step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.clamp(torch.round(z / step) * step, -TOP, TOP) * unit


def _least(top):
    """The least whole e with top <= 448 2^e, by trying all."""
    every = torch.arange(-RANGE, RANGE + 1, device=top.device)
    fits = top[..., None] <= TOP * torch.exp2(every.double())
    return torch.where(fits.any(-1), fits.int().argmax(-1) - RANGE, RANGE)


def _history(s, r, codes, exps, n):
    """Tokens 0 .. n - 1 of request r as float64 [n][hkv][d], and their exponents [n][hkv]."""
    pages = s["table"][r, :-(-n // s["case"]["page"])].long()
    e = exps[pages].transpose(1, 2).reshape(-1, exps.shape[1]).long().repeat_interleave(BLOCK, 0)[:n]
    x = _take(codes, pages).float().transpose(1, 2).reshape(-1, codes.shape[1], codes.shape[3])[:n]
    return x.double() * torch.exp2(e.double())[..., None], e


def exact(case, seed):
    s = prepare(case, seed)
    hkv, d = case["hkv"], case["d"]
    g = case["hq"] // hkv
    rows, kv = _lengths(case)
    start = np.cumsum(rows) - rows
    if case["op"] == "norm":
        return _turned(case, s, s["q"], s["qw"]), _turned(case, s, s["k"], s["kw"])
    if case["op"] in ("append", "read"):
        new = {}
        if case["op"] == "append":
            new = {"k": _turned(case, s, s["k"], s["kw"]), "v": s["v"].double()}
        found = {"k": [], "v": []}
        for r in range(case["requests"]):
            n, m, a = int(kv[r]), int(rows[r]), int(start[r])
            for name in "kv":
                if case["op"] == "read":
                    x, _ = _history(s, r, s[name + "_cache"], s[name + "_exp"], n)
                    found[name].append(x[n - m:])
                    continue
                fill = (n - m) % BLOCK
                x, e = _history(s, r, s[name + "_cache"], s[name + "_exp"], n - m)
                y = torch.cat((x[n - m - fill:], new[name][a:a + m]))
                short = -len(y) % BLOCK
                y = torch.cat((y, y.new_zeros(short, hkv, d))).view(-1, BLOCK, hkv, d)
                z = y.clone()
                if fill:
                    z[0, :fill] = 0.0
                least = _least(z.abs().amax(-1).amax(1))
                if fill:
                    least[0] = torch.maximum(least[0], e[-1])
                found[name].append(_on_grid(y, least[:, None, :, None]).view(-1, hkv, d)[:fill + m])
        back = torch.cat(found["k"]), torch.cat(found["v"])
        return back if case["op"] == "read" else (_turned(case, s, s["q"], s["qw"]),) + back
    if work(case)["flops"] > 6.0e12:
        return None
    o = torch.zeros(s["t"], case["hq"], d, device="cuda", dtype=torch.float64)
    lse = torch.full((s["t"], case["hq"]), -math.inf, device="cuda", dtype=torch.float64)
    for r in range(case["requests"]):
        n, m, a = int(kv[r]), int(rows[r]), int(start[r])
        seen = torch.arange(n, device="cuda") < (torch.arange(m, device="cuda") + n - m + 1)[:, None]
        keys, _ = _history(s, r, s["k_cache"], s["k_exp"], n)
        values, _ = _history(s, r, s["v_cache"], s["v_exp"], n)
        for h in range(hkv):
            k, v = keys[:, h].contiguous(), values[:, h].contiguous()
            for j in range(h * g, h * g + g):
                x = s["q"][a:a + m, j].double() @ k.t() / math.sqrt(d)
                x = torch.where(seen, x, -math.inf)
                z = torch.logsumexp(x, -1)
                o[a:a + m, j], lse[a:a + m, j] = torch.exp(x - z[:, None]) @ v, z
    return o, lse
