"""What is measured of the attention-layer operators that serve beside the GDN core.

Three operators, for the softmax-attention layers that a hybrid stack puts
between its Gated DeltaNet layers:

  rope    rotary positions on query and key rows, one position axis or
          several (time, height, width), forward and inverse (the gradient);
  append  keys rotated and written with their values into a paged cache, the
          queries rotated on the way;
  attn    causal attention of a step's query rows over the paged cache, for
          requests of which groups share leading pages.

``run`` computes the plain form in 32 bits with elementary torch operations,
or, where ``own`` is true, calls the framework's entry points. ``exact`` is
the definition in 64 bits, request by request.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------- cases

def _case(op, name, **kw):
    c = {"name": name, "op": op, "dtype": "bf16", "hq": 32, "hkv": 8, "d": 128, "rd": 128,
         "axes": 1, "interleaved": False, "inverse": False, "requests": 1, "rows_min": 1,
         "rows_max": 1, "kv_min": 0, "kv_max": 0, "page": 64, "groups": 0, "shared": 0,
         "base": 1.0e6, "first": 0, "short": 0, "mix": 1}
    c.update(kw)
    return c


def listed():
    return [
        # one decode step's rows of 64 requests, rotary on a quarter of wide heads
        _case("rope", "rope_decode", requests=64, hq=16, hkv=2, d=256, rd=64, first=120000),
        # image and video patches of a vision tower: three axes, narrow heads of an odd width
        _case("rope", "rope_video", requests=4, rows_min=6000, rows_max=9000, hq=16, hkv=16, d=80,
              rd=80, axes=3, base=1.0e4),
        # a training step's gradients in 32 bits go back through the rotation
        _case("rope", "rope_grad", requests=4, rows_min=2048, rows_max=2048, dtype="f32",
              inverse=True, interleaved=True),
        # the smallest step: one request, one new token
        _case("append", "append_one", kv_min=776, kv_max=776),
        # speculative candidates and short prompts packed into one step, three axes
        _case("append", "append_mixed", requests=40, rows_min=8, rows_max=400,
              kv_max=4000, hq=16, hkv=2, d=256, rd=64, axes=3, page=16, short=80),
        # long prompts enter the cache at once
        _case("append", "append_prompt", requests=4, rows_min=8192, rows_max=8192,
              dtype="f16", page=128),
        # the smallest attention call: one token of one request, a few hundred keys
        _case("attn", "attn_one", kv_min=512, kv_max=512),
        # a decode batch of ragged lengths with nothing shared
        _case("attn", "attn_decode", requests=64, kv_max=16383, page=16),
        # a decode batch behind one long instruction: wide heads, eight queries to a key head
        _case("attn", "attn_shared", requests=64, hq=16, hkv=2, d=256, rd=64,
              kv_max=1023, groups=1, shared=16384),
        # speculative verification (1 + 7 rows) in four groups, each behind its own prefix
        _case("attn", "attn_verify", requests=64, rows_min=8, rows_max=8, dtype="f16",
              kv_max=900, groups=4, shared=4096, page=32),
        # prompt pieces over a shared document: long on both sides, so compute counts
        _case("attn", "attn_prompt", requests=4, rows_min=1500, rows_max=2048, kv_max=512,
              groups=1, shared=8192),
        # many narrow-headed requests that branch from one very long prefix
        _case("attn", "attn_branch", requests=96, hq=32, hkv=4, d=64, rd=64, kv_max=300,
              groups=1, shared=49152, page=128),
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
        op = rng.choice(["rope", "append", "attn", "attn", "attn"])
        hkv = rng.choice([1, 2, 4, 8])
        g = rng.choice([1, 2, 3, 4, 6, 8, 16])
        c = _case(op, "drawn", hkv=hkv, hq=hkv * g, dtype=rng.choice(["bf16", "bf16", "f16"]),
                  page=rng.choice([16, 32, 64, 128]), mix=rng.randrange(1 << 20))
        if c["hq"] > 64:
            continue
        if op == "rope":
            c["d"] = rng.choice([64, 72, 80, 96, 128, 256])
            c["rd"] = rng.choice([c["d"], c["d"], c["d"] // 2])
            c["dtype"] = rng.choice(["bf16", "f16", "f32"])
            c["requests"] = _log(rng, 1, 64)
            c["rows_min"] = c["rows_max"] = 1
            if rng.random() < 0.7:
                c["rows_max"] = _log(rng, 1, 16384 // c["requests"])
                c["rows_min"] = max(1, c["rows_max"] // 3)
            c["inverse"] = rng.random() < 0.4
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
                c["rows_max"] = _log(rng, 9, 8192 if op == "append" else 2048)
                c["rows_min"] = rng.randint(1, c["rows_max"])
            c["kv_max"] = _log(rng, 1, 24000)
            c["kv_min"] = rng.randint(0, c["kv_max"])
            if op == "attn" and rng.random() < 0.6:
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
        if t <= 40000 and _cost(c) <= most and (op == "rope" or pad < 4.0e10):
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


def work(case):
    e, d, hq, hkv = SIZE[case["dtype"]], case["d"], case["hq"], case["hkv"]
    rows, kv = _lengths(case)
    t = int(rows.sum())
    if case["op"] == "rope":
        # every row in and out, and its positions; six operations a rotated pair of values
        return {"bytes": 2.0 * t * (hq + hkv) * d * e + 4.0 * t * case["axes"],
                "flops": 3.0 * t * (hq + hkv) * case["rd"]}
    if case["op"] == "append":
        return {"bytes": 2.0 * t * (hq + 2 * hkv) * d * e + 4.0 * t * case["axes"],
                "flops": 3.0 * t * (hq + hkv) * case["rd"]}
    # each key and value once for all that share it; each row in, its output and its lse out
    shared = _shared_pages(case) * case["page"]
    keys = float((kv - shared).sum()) + float(shared * case["groups"])
    pairs = float((rows * kv - rows * (rows - 1) // 2).sum())
    return {"bytes": 2.0 * keys * hkv * d * e + 2.0 * t * hq * d * e + 4.0 * t * hq,
            "flops": 4.0 * pairs * hq * d}


# ------------------------------------------------------------------ inputs

def _positions(case, rows, kv, gen):
    """int32 [axes][rows]: the place of each row in its sequence; on three axes, of a
    video's patches (a frame of 24 x 32), each axis with its own."""
    t = np.concatenate([np.arange(b - a, b) for a, b in zip(rows, kv)]) if len(rows) else np.zeros(0)
    t = t + case["first"]
    if case["axes"] == 1:
        p = t[None]
    else:
        p = np.stack([case["first"] + t // 768, (t // 32) % 24 + t // 768, t % 32 + t // 768])
    p = torch.from_numpy(p.astype(np.int32)).cuda()
    # new inputs for each seed: the whole step somewhere else
    return (p + torch.randint(0, 64, (1,), generator=gen, device="cuda", dtype=torch.int32)).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    dt, d, hq, hkv, ps = TYPES[case["dtype"]], case["d"], case["hq"], case["hkv"], case["page"]
    rows, kv = _lengths(case)
    t, n = int(rows.sum()), case["requests"]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dt)

    def i32(v):
        return torch.from_numpy(np.ascontiguousarray(v, dtype=np.int32)).cuda()

    s = {"case": dict(case), "t": t}
    half = case["rd"] // 2
    s["inv_freq"] = (1.0 / case["base"] ** (torch.arange(half, device="cuda", dtype=torch.float64)
                                            / half)).float()
    # time, height and width take turns over the frequencies
    s["axis"] = i32(np.arange(half) % case["axes"])
    s["pos"] = _positions(case, rows, kv, gen)
    # the projections write q, k and v of a row side by side
    qkv = randn(t, hq + 2 * hkv, d)
    s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    s["q_out"] = torch.empty(t, hq, d, device="cuda", dtype=dt)
    if case["op"] == "rope":
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
        s["k_cache"], s["v_cache"] = randn(pool, hkv, ps, d), randn(pool, hkv, ps, d)
        s["row_start"], s["row_len"] = i32(np.cumsum(rows) - rows), i32(rows)
        s["kv_len"] = i32(kv)
        s["row_req"] = i32(np.repeat(np.arange(n), rows)).long()
        s["row_t"] = i32(np.concatenate([np.arange(a) for a in rows])).long()
        if case["groups"]:
            a, c = _groups(case)
            s["group"] = (i32(a), i32(c), i32(np.full(case["groups"], shared)))
        s["o"], s["lse"] = torch.empty_like(s["q_out"]), torch.empty(t, hq, device="cuda")
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
    s["rope"] = gdn.make_rope(case["rd"], s["inv_freq"], s["pos"], axis=s["axis"],
                              interleaved=case["interleaved"])
    if case["op"] == "rope":
        return
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    s["batch"] = gdn.make_kv_batch(case["requests"], s["t"], int(rows.max()),
                                   s["k_cache"].shape[0], s["row_start"], s["row_len"],
                                   s["kv_len"], s["table"], *s.get("group", ()))
    if case["op"] == "attn":
        nbytes = gdn.gdn_attn_plan_bytes(s["dims"], s["batch"])
        s["plan"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        nbytes = gdn.gdn_attn_workspace_bytes(s["dims"], s["batch"])
        s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        gdn.gdn_attn_plan(s["dims"], s["batch"], s["plan"], s["plan"].numel(), s["status"])


# --------------------------------------------------------------- plain form

def _cos_sin(s):
    """cos and sin [rows][rotary_dim / 2] of position times frequency. The product's
    rounding error is carried beside it (both factors split into 12-bit halves, whose
    products are exact), so that far positions keep the precision of near ones."""
    p = s["pos"][s["axis"].long()].t().float()
    f = s["inv_freq"][None]
    big = f * 4097.0
    fh = big - (big - f)
    fl = f - fh
    ph = torch.floor(p / 4096.0) * 4096.0
    pl = p - ph
    a = p * f
    e = ((ph * fh - a) + ph * fl + pl * fh) + pl * fl
    ca, sa, ce, se = torch.cos(a), torch.sin(a), torch.cos(e), torch.sin(e)
    return ca * ce - sa * se, sa * ce + ca * se


def _rotate(s, x, cos, sin):
    case = s["case"]
    rd = case["rd"]
    sin = -sin if case["inverse"] else sin
    cos, sin = cos[:, None], sin[:, None]
    y = x.float()
    r, rest = y[..., :rd], y[..., rd:]
    if case["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r[..., :rd // 2], r[..., rd // 2:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((r, rest), -1).to(x.dtype)


def _plain_append(s):
    cos, sin = _cos_sin(s)
    at = s["kv_len"].long()[s["row_req"]] - s["row_len"].long()[s["row_req"]] + s["row_t"]
    ps = s["case"]["page"]
    page, slot = s["table"].long()[s["row_req"], at // ps], at % ps
    s["k_cache"][page, :, slot] = _rotate(s, s["k"], cos, sin)
    s["v_cache"][page, :, slot] = s["v"]
    return _rotate(s, s["q"], cos, sin), s["k_cache"], s["v_cache"]


def _plain_attn(s):
    case = s["case"]
    n, hkv, d, ps = case["requests"], case["hkv"], case["d"], case["page"]
    g, tm = case["hq"] // hkv, case["rows_max"]
    table = s["table"].long()
    width = table.shape[1] * ps
    k = s["k_cache"][table].transpose(1, 2).reshape(n, hkv, width, d).float()
    v = s["v_cache"][table].transpose(1, 2).reshape(n, hkv, width, d).float()
    step = torch.arange(tm, device="cuda")
    row = (s["row_start"].long()[:, None] + step).clamp_(max=s["t"] - 1)
    q = s["q"][row].float().view(n, tm, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, g * tm, d)
    score = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    last = (s["kv_len"].long() - s["row_len"].long())[:, None] + step  # the row's own key
    seen = torch.arange(width, device="cuda") <= last[..., None]
    score.view(n, hkv, g, tm, width).masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    score = score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    o = torch.matmul(score, v) / total
    lse = (top + total.log()).squeeze(-1)
    o = o.view(n, hkv, g, tm, d).permute(0, 3, 1, 2, 4).reshape(n, tm, hkv * g, d)
    lse = lse.view(n, hkv, g, tm).permute(0, 3, 1, 2).reshape(n, tm, hkv * g)
    return o[s["row_req"], s["row_t"]].to(s["q"].dtype), lse[s["row_req"], s["row_t"]]


def run(s):
    op = s["case"]["op"]
    if own:
        gdn = s["gdn"]
        if op == "rope":
            gdn.gdn_rope(s["dims"], s["rope"], s["q"], s["q_out"], s["k"], s["k_out"],
                         inverse=s["case"]["inverse"])
            return s["q_out"], s["k_out"]
        if op == "append":
            gdn.gdn_kv_append(s["dims"], s["batch"], s["rope"], s["q"], s["k"], s["v"], s["q_out"],
                              s["k_cache"], s["v_cache"], s["status"])
            return s["q_out"], s["k_cache"], s["v_cache"]
        gdn.gdn_attn(s["dims"], s["batch"], s["plan"], s["q"], s["k_cache"], s["v_cache"], s["o"],
                     s["lse"], s["workspace"], s["workspace"].numel(), s["status"])
        return s["o"], s["lse"]
    if op == "rope":
        cos, sin = _cos_sin(s)
        return _rotate(s, s["q"], cos, sin), _rotate(s, s["k"], cos, sin)
    return _plain_append(s) if op == "append" else _plain_attn(s)


# ------------------------------------------------------------- in 64 bits

def _turned(case, x, pos, axis, inv_freq):
    """The rotation as complex numbers: pair j of row i times e^{+-i position frequency}."""
    rd = case["rd"]
    angle = pos.double()[axis.long()].t() * inv_freq.double()
    turn = torch.polar(torch.ones_like(angle), -angle if case["inverse"] else angle)[:, None]
    y = x.double().clone()
    if case["interleaved"]:
        z = torch.view_as_complex(y[..., :rd].reshape(*y.shape[:-1], rd // 2, 2).contiguous()) * turn
        y[..., :rd] = torch.view_as_real(z).reshape(*y.shape[:-1], rd)
    else:
        z = torch.complex(y[..., :rd // 2].contiguous(), y[..., rd // 2:rd].contiguous()) * turn
        y[..., :rd // 2], y[..., rd // 2:rd] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    ps, hkv = case["page"], case["hkv"]
    g = case["hq"] // hkv
    rows, kv = _lengths(case)
    start = np.cumsum(rows) - rows
    if case["op"] == "rope":
        return tuple(_turned(case, s[x], s["pos"], s["axis"], s["inv_freq"]) for x in "qk")
    if case["op"] == "append":
        q, k = (_turned(case, s[x], s["pos"], s["axis"], s["inv_freq"]) for x in "qk")
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        for r in range(case["requests"]):
            a, b = int(start[r]), int(start[r] + rows[r])
            at = torch.arange(int(kv[r] - rows[r]), int(kv[r]), device="cuda")
            page = s["table"][r].long()[at // ps]
            kc[page, :, at % ps], vc[page, :, at % ps] = k[a:b], s["v"][a:b].double()
        return q, kc, vc
    if work(case)["flops"] > 6.0e12:
        return None
    o = torch.zeros(s["t"], case["hq"], case["d"], device="cuda", dtype=torch.float64)
    lse = torch.full((s["t"], case["hq"]), -math.inf, device="cuda", dtype=torch.float64)
    for r in range(case["requests"]):
        n, m, a = int(kv[r]), int(rows[r]), int(start[r])
        pages = s["table"][r, :-(-n // ps)].long()
        seen = torch.arange(n, device="cuda") < (torch.arange(m, device="cuda") + n - m + 1)[:, None]
        for h in range(hkv):
            k = s["k_cache"][pages, h].reshape(-1, case["d"])[:n].double()
            v = s["v_cache"][pages, h].reshape(-1, case["d"])[:n].double()
            for j in range(h * g, h * g + g):
                x = s["q"][a:a + m, j].double() @ k.t() / math.sqrt(case["d"])
                x = torch.where(seen, x, -math.inf)
                z = torch.logsumexp(x, -1)
                o[a:a + m, j], lse[a:a + m, j] = torch.exp(x - z[:, None]) @ v, z
    return o, lse
