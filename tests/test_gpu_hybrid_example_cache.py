"""The hybrid example's prompt lies in the shared pages as it should: keys rotated at the positions
0, 1, ..., values as they were projected."""
import pytest
import torch

from tests.test_gpu_attn_layer import check_rotated, rotate64
from tests.test_gpu_hybrid_example import load

pytestmark = pytest.mark.gpu


def test_cached_prompt(monkeypatch):
    m = load()
    calls = []
    append = m.gdn.gdn_kv_append

    def recorded(dims, batch, rope, q, k, v, *rest, **kw):
        calls.append((k.clone(), v.clone()))
        return append(dims, batch, rope, q, k, v, *rest, **kw)

    monkeypatch.setattr(m.gdn, "gdn_kv_append", recorded)
    pages = 7
    _, _, attn, table, _, inv_freq = m.main(requests=5, prompt_pages=pages, steps=2)
    k, v = calls[0]
    n = pages * m.PAGE
    assert k.shape[0] == n
    pos = torch.arange(n, device="cuda", dtype=torch.int32)[None]
    axis = torch.zeros(m.ROT // 2, dtype=torch.int32, device="cuda")
    want, r = rotate64(k, pos, axis, inv_freq, m.ROT, False, False)
    shared = table[0, :pages].long()
    kept_k, kept_v = (c[shared].transpose(1, 2).reshape(n, m.HKV, m.D)
                      for c in (attn.cache.k, attn.cache.v))
    check_rotated(kept_k, want, r)
    assert torch.equal(kept_v, v)
