"""A few decode steps of a small hybrid stack on random weights: three Gated
DeltaNet layers, then one softmax-attention layer, as hybrid models alternate
them. Requests of one group continue the same prompt, whose pages they share.

Per step the caller plans the attention once; per layer it makes one call for
a GDN layer (gdn_decode) and two for an attention layer (gdn_kv_append, which
rotates q and k on the way, and gdn_attn). With --bits 8 the attention layer norms
its queries and keys and keeps them and its values in 8 bits (gdn_kv8_append and
gdn_kv8_attn).

    python examples/hybrid_step.py [--bits 8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_linear_14_gb300 as gdn  # noqa: E402
from gated_deltanet_linear_14_gb300.pages import Kv8Cache, KvCache, PagePool  # noqa: E402

HIDDEN, GDN_LAYERS = 1024, 3
HK, HV, DG = 4, 8, 128             # GDN heads and head dimension
HQ, HKV, D, ROT, PAGE = 8, 2, 256, 64, 64   # attention heads, a quarter of each rotated


def i32(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


class Linear:
    def __init__(self, n_in, n_out, g):
        self.w = (torch.randn(n_in, n_out, device="cuda", generator=g) / n_in ** 0.5).bfloat16()

    def __call__(self, x):
        return x @ self.w


class GdnLayer:
    def __init__(self, requests, g):
        self.dims = gdn.make_dims(HK, HV, DG, DG, W=4, Kc=0)
        self.pool = PagePool(self.dims, requests)
        self.A_log = torch.rand(HV, device="cuda", generator=g) * 2 - 1
        self.dt_bias = torch.rand(HV, device="cuda", generator=g) - 0.5
        self.params = gdn.make_params(self.A_log, self.dt_bias)
        self.conv_w = (torch.rand(self.dims.C, 4, device="cuda", generator=g) - 0.5).bfloat16()
        self.inp, self.gates = Linear(HIDDEN, self.dims.C, g), Linear(HIDDEN, 2 * HV, g)
        self.out = Linear(HV * DG, HIDDEN, g)

    def step(self, x, batch, status):
        ab = self.gates(x)
        a, b = ab[:, :HV].contiguous(), ab[:, HV:].contiguous()
        o = torch.empty(x.shape[0], HV, DG, device="cuda", dtype=torch.bfloat16)
        gdn.gdn_decode(self.dims, batch, self.params, self.inp(x), self.conv_w, a, b, o,
                       self.pool.buf, status)
        return x + self.out(o.flatten(1))


class AttentionLayer:
    def __init__(self, pages, g):
        self.dims = gdn.make_attn_dims(HQ, HKV, D, PAGE)
        self.cache = KvCache(self.dims, pages)
        self.qkv, self.out = Linear(HIDDEN, (HQ + 2 * HKV) * D, g), Linear(HQ * D, HIDDEN, g)

    def rows(self, x):
        qkv = self.qkv(x).view(-1, HQ + 2 * HKV, D)
        return qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]

    def step(self, x, batch, rope, plan, workspace, status):
        q, k, v = self.rows(x)
        q_rot = torch.empty(x.shape[0], HQ, D, device="cuda", dtype=torch.bfloat16)
        o = torch.empty_like(q_rot)
        gdn.gdn_kv_append(self.dims, batch, rope, q, k, v, q_rot, self.cache.k, self.cache.v,
                          status)
        gdn.gdn_attn(self.dims, batch, plan, q_rot, self.cache.k, self.cache.v, o, None,
                     workspace, workspace.numel(), status)
        return x + self.out(o.flatten(1))

    def plan_for(self, batch, status):
        plan, workspace = (torch.empty(size(self.dims, batch), dtype=torch.uint8, device="cuda")
                           for size in (gdn.gdn_attn_plan_bytes, gdn.gdn_attn_workspace_bytes))
        gdn.gdn_attn_plan(self.dims, batch, plan, plan.numel(), status)
        return plan, workspace


class AttentionLayer8(AttentionLayer):
    """Queries and keys normed head by head, keys and values kept in 8 bits."""

    def __init__(self, pages, g):
        super().__init__(pages, g)
        self.cache = Kv8Cache(self.dims, pages)
        self.q_norm, self.k_norm = (0.1 * torch.randn(D, device="cuda", generator=g)
                                    for _ in range(2))
        self.norm = gdn.make_head_norm(self.q_norm, self.k_norm, offset=1.0)

    def step(self, x, batch, rope, plan, workspace, status):
        q, k, v = self.rows(x)
        q_rot = torch.empty(x.shape[0], HQ, D, device="cuda", dtype=torch.bfloat16)
        o = torch.empty_like(q_rot)
        gdn.gdn_kv8_append(self.dims, batch, self.norm, rope, q, k, v, q_rot, self.cache.codes,
                           status)
        gdn.gdn_kv8_attn(self.dims, batch, plan, q_rot, self.cache.codes, o, None, workspace,
                         workspace.numel(), status)
        return x + self.out(o.flatten(1))

    def plan_for(self, batch, status):
        plan, workspace = (torch.empty(size(self.dims, batch), dtype=torch.uint8, device="cuda")
                           for size in (gdn.gdn_kv8_attn_plan_bytes,
                                        gdn.gdn_kv8_attn_workspace_bytes))
        gdn.gdn_kv8_attn_plan(self.dims, batch, plan, plan.numel(), status)
        return plan, workspace


def main(requests=16, prompt_pages=20, steps=4, seed=0, bits=16):
    """The hidden states of the last step, and the attention layer with its page table and
    lengths (for checks)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    R, prompt = requests, prompt_pages * PAGE
    gdn_layers = [GdnLayer(R, g) for _ in range(GDN_LAYERS)]
    attn = (AttentionLayer8 if bits == 8 else AttentionLayer)(prompt_pages + R, g)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    inv_freq = 1.0 / 1e6 ** (torch.arange(ROT // 2, device="cuda").float() / (ROT // 2))

    # every request: the prompt's pages, then one page of its own
    table = torch.cat([torch.arange(prompt_pages).repeat(R, 1),
                       prompt_pages + torch.arange(R)[:, None]], 1).int().cuda()
    # the prompt enters the shared pages once, as one request's rows
    x = torch.randn(prompt, HIDDEN, device="cuda", generator=g).bfloat16()
    maps = (i32([0]), i32([prompt]), i32([prompt]), table)
    rope = gdn.make_rope(ROT, inv_freq, torch.arange(prompt, device="cuda", dtype=torch.int32))
    first = gdn.make_kv_batch(1, prompt, prompt, attn.cache.num_pages, *maps)
    attn.step(x, first, rope, *attn.plan_for(first, status), status)

    # then R requests go on from it, one token a step
    ones, rows, group = i32([1] * R), i32(range(R)), (i32([0]), i32([R]), i32([prompt_pages]))
    fresh, goes_on = i32([gdn.GDN_REQ_FRESH] * R), i32([0] * R)
    x = torch.randn(R, HIDDEN, device="cuda", generator=g).bfloat16()
    for t in range(steps):
        kv_len = i32([prompt + t + 1] * R)
        gdn_batch = gdn.make_batch(R, R, 1, R, rows, ones, rows, goes_on if t else fresh)
        kv_batch = gdn.make_kv_batch(R, R, 1, attn.cache.num_pages, rows, ones, kv_len, table,
                                     *group)
        positions = kv_len - 1
        rope = gdn.make_rope(ROT, inv_freq, positions)
        plan, workspace = attn.plan_for(kv_batch, status)  # for all attention layers
        for layer in gdn_layers:
            x = layer.step(x, gdn_batch, status)
        before = x
        x = attn.step(x, kv_batch, rope, plan, workspace, status)
    gdn.raise_on_status(status, "hybrid step")
    return before, x, attn, table, kv_len, inv_freq


if __name__ == "__main__":
    parser = argparse.ArgumentParser()
    parser.add_argument("--bits", type=int, choices=(8, 16), default=16, help="of the key/value cache")
    out = main(bits=parser.parse_args().bits)[1]
    print(f"hybrid step ok: {out.shape[0]} requests, |x| = {out.float().norm().item():.3f}")
