"""The hybrid example with an 8-bit cache: norms, rotation, append, plan and attention as they are
used together. Its last attention layer equals the plain form on what its cache stands for, and the
cached prompt is what was projected, normed, rotated and rounded once."""
import pytest
import torch

from tests.kv8_util import Blocks, grid_step, normed, partners, rotated
from tests.test_gpu_hybrid_example import load
from gated_deltanet_linear_14_gb300.pages import Kv8Cache

pytestmark = pytest.mark.gpu


def test_hybrid_step_8_bits(monkeypatch):
    m = load()
    calls = []
    append = m.gdn.gdn_kv8_append

    def recorded(dims, batch, norm, rope, q, k, v, *rest, **kw):
        calls.append((k.clone(), v.clone()))
        return append(dims, batch, norm, rope, q, k, v, *rest, **kw)

    monkeypatch.setattr(m.gdn, "gdn_kv8_append", recorded)
    pages, R = 7, 5
    before, after, attn, table, kv_len, inv_freq = m.main(requests=R, prompt_pages=pages, steps=3,
                                                          bits=8)
    assert bool(torch.isfinite(after.float()).all())
    # the prompt in the shared pages
    k, v = calls[0]
    n, shared = pages * m.PAGE, table[0, :pages].long()

    def stored(codes, exps):
        x = Kv8Cache.values(codes.view(torch.uint8)[shared].view(codes.dtype), exps[shared])
        return (x.double().transpose(1, 2).reshape(n, m.HKV, m.D),
                exps[shared].long().transpose(1, 2).reshape(-1, m.HKV))

    want = Blocks(m.HKV, m.D)
    want.append(v.double(), 0)
    x, e = stored(attn.cache.v, attn.cache.v_exp)
    assert torch.equal(x, want.x) and torch.equal(e, want.e)
    y = normed(k, attn.k_norm, 1e-6, 1.0)
    pos = torch.arange(n, device="cuda", dtype=torch.int32)
    turned = rotated(y, m.ROT, inv_freq, pos)
    x, e = stored(attn.cache.k, attn.cache.k_exp)
    unit = torch.exp2(e.double()).repeat_interleave(16, 0)[..., None]
    room = grid_step(turned / unit) / 2 * unit * (1 + 1e-9) + partners(y, m.ROT, False) * 2.0 ** -18
    assert bool(((x - turned).abs() <= room).all())

    # the last step's attention
    G = m.HQ // m.HKV
    q, _, _ = attn.rows(before)
    q = rotated(normed(q, attn.q_norm, 1e-6, 1.0), m.ROT, inv_freq, kv_len - 1).bfloat16().double()
    o = torch.empty(R, m.HQ, m.D, dtype=torch.float64, device="cuda")
    for r in range(R):
        t, c = table[r].long(), int(kv_len[r])
        keys, values = (
            Kv8Cache.values(x.view(torch.uint8)[t].view(x.dtype), e[t]).double().transpose(0, 1)
            .reshape(m.HKV, -1, m.D)[:, :c] for x, e in ((attn.cache.k, attn.cache.k_exp),
                                                         (attn.cache.v, attn.cache.v_exp)))
        for h in range(m.HQ):
            p = torch.softmax(keys[h // G] @ q[r, h] / m.D ** 0.5, 0)
            o[r, h] = p @ values[h // G]
    want = before.double() + o.flatten(1) @ attn.out.w.double()
    # as for 16 bits (roundings of o, the projection's and the sum's results, and of q), with p
    # within 2^-7: one half more
    bound = 5 * 2.0 ** -8 * want.abs().clamp_min(want.pow(2).mean().sqrt().item())
    assert bool(((after.double() - want).abs() <= bound).all())
