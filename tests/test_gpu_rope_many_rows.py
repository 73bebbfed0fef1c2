"""A rotation of as many rows as an int32 counts."""
import math

import pytest
import torch

import gated_deltanet_linear_14_gb300 as gdn

pytestmark = pytest.mark.gpu


def test_nearly_2_31_rows():
    rows = (1 << 31) - 1
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 20 GB")
    pos = torch.empty(rows, dtype=torch.int32, device="cuda").fill_(3)
    q = torch.empty(rows, 1, 2, dtype=torch.float16, device="cuda").fill_(1)
    freq = torch.tensor([0.5], device="cuda")
    gdn.gdn_rope(gdn.make_attn_dims(1, 1, 2, 16, io=gdn.GDN_F16), gdn.make_rope(2, freq, pos), q, q)
    want = torch.tensor([math.cos(1.5) - math.sin(1.5), math.cos(1.5) + math.sin(1.5)],
                        device="cuda").half()
    for part in q.split(1 << 28):
        assert bool(((part[:, 0] - want).abs() <= 2.0 ** -10).all())
