"""What the Python calls of the attention layers do with tensors that do not fit: they are refused
before anything is launched. The tensors here lie in host memory, which no call gets to read: where
a call passes the checks it stops at the missing device."""
import gc
import weakref

import pytest
import torch

import gated_deltanet_linear_14_gb300 as gdn
from gated_deltanet_linear_14_gb300 import build as gbuild

INVALID = gdn.CODES["GDN_ERR_INVALID_ARG"]


@pytest.fixture(scope="module", autouse=True)
def lib():
    gbuild.build()
    return gdn.load_library()


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_structures_keep_their_tensors():
    """A structure holds addresses: a tensor made in the call itself must live as long."""
    def made(make, *args, **kw):
        refs = []

        def held(t):
            refs.append(weakref.ref(t))
            return t

        s = make(*[held(a()) if callable(a) else a for a in args],
                 **{k: held(a()) for k, a in kw.items()})
        gc.collect()
        assert all(r() is not None for r in refs)
        del s
        gc.collect()
        assert all(r() is None for r in refs)

    made(gdn.make_rope, 64, lambda: torch.ones(32), lambda: i32(3, 5), axis=lambda: i32(32))
    made(gdn.make_kv_batch, 4, 4, 1, 9, *[lambda: i32(4)] * 3, lambda: i32(4, 2),
         group_start=lambda: i32(1), group_len=lambda: i32(1), group_pages=lambda: i32(1))
