"""The wait that the attention kernel's warps make: it gives up after its limit and leaves word, by
which the waits after it end at once (each of them alone would take ten seconds here)."""
import time

import pytest
import torch

import gated_deltanet_linear_14_gb300 as gdn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("limit", [1_000_000, 200_000_000])
def test_a_wait_that_gave_up_ends_the_next(limit):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_check_bounded_wait(1000, status)  # (loads the kernel)
    torch.cuda.synchronize()
    status.zero_()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    gdn.gdn_check_bounded_wait(limit, status)
    torch.cuda.synchronize()
    waited = time.perf_counter() - t0
    assert int(status.item()) == gdn.CODES["GDN_DEV_TIMEOUT"]
    assert 0.9e-9 * limit <= waited < 1e-9 * limit + 1.0, waited
