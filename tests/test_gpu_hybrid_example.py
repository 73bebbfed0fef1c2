"""The hybrid example (GDN layers and an attention layer in one step) runs through the public
calls, and its last attention layer equals the plain form on the cache that it left."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load():
    spec = importlib.util.spec_from_file_location("hybrid_step",
                                                  os.path.join(ROOT, "examples/hybrid_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_hybrid_step():
    m = load()
    before, after, attn, table, kv_len, inv_freq = m.main(requests=5, prompt_pages=7, steps=3)
    assert bool(torch.isfinite(after.float()).all())
    G = m.HQ // m.HKV
    q, _, _ = attn.rows(before)
    angle = (kv_len - 1).double()[:, None] * inv_freq.double()
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    q = q.double().clone()
    a, b = q[..., :m.ROT // 2].clone(), q[..., m.ROT // 2:m.ROT].clone()
    q[..., :m.ROT // 2], q[..., m.ROT // 2:m.ROT] = a * c - b * s, b * c + a * s
    q = q.bfloat16().double()  # as the call stores it
    o = torch.empty(5, m.HQ, m.D, dtype=torch.float64, device="cuda")
    for r in range(5):
        n = int(kv_len[r])
        k, v = (x[table[r].long()].transpose(0, 1).reshape(m.HKV, -1, m.D)[:, :n].double()
                for x in (attn.cache.k, attn.cache.v))
        for h in range(m.HQ):
            p = torch.softmax(k[h // G] @ q[r, h] / m.D ** 0.5, 0)
            o[r, h] = p @ v[h // G]
    want = before.double() + o.flatten(1) @ attn.out.w.double()
    # bf16 roundings of p, o and the projection's and the sum's results: 2^-8 each of terms
    # of the hidden state's size
    bound = 4 * 2.0 ** -8 * want.abs().clamp_min(want.pow(2).mean().sqrt().item())
    assert bool(((after.double() - want).abs() <= bound).all())
