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


BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def rows(n, heads, dim=64, dtype=BF):
    return torch.zeros(n, heads, dim, dtype=dtype)


def code_of(call, *args, **kw):
    with pytest.raises(gdn.GdnError) as e:
        call(*args, stream=0, **kw)
    return e.value.code


def rope_code(q, q_out, k=None, k_out=None, dims=None, positions=None):
    dims = dims or gdn.make_attn_dims(4, 2, 64, 16)
    positions = i32((q if q is not None else k).shape[0]) if positions is None else positions
    return code_of(gdn.gdn_rope, dims, gdn.make_rope(64, torch.ones(32), positions), q, q_out, k,
                   k_out)


@pytest.mark.skipif(torch.cuda.is_available(), reason="host memory is passed on to the launch")
def test_rope_rows_that_fit_reach_the_launch():
    assert rope_code(rows(5, 4), rows(5, 4), rows(5, 2), rows(5, 2)) != INVALID
    assert rope_code(rows(5, 4), rows(9, 4)) != INVALID                 # an output with more rows
    assert rope_code(rows(5, 6)[:, :4], rows(5, 4)) != INVALID          # a slice of the heads
    assert rope_code(rows(1, 6), rows(1, 4)) != INVALID                 # more heads than are turned


def test_rope_rows_that_do_not_fit_are_refused():
    q, k = rows(5, 4), rows(5, 2)
    assert rope_code(q, rows(4, 4)) == INVALID                          # fewer rows out than in
    assert rope_code(q, q, rows(4, 2), k) == INVALID                    # k shorter than q
    assert rope_code(q, q, rows(6, 2), rows(6, 2)) == INVALID           # and longer
    assert rope_code(q, q, k, rows(4, 2)) == INVALID
    assert rope_code(rows(5, 3), q) == INVALID                          # fewer heads
    assert rope_code(q, rows(5, 3)) == INVALID
    assert rope_code(rows(5, 4, 32), q) == INVALID                      # another width
    assert rope_code(rows(5, 4, dtype=F32), q) == INVALID               # another type
    assert rope_code(q, rows(5, 4, dtype=HF)) == INVALID
    assert rope_code(rows(5, 4, 128)[..., ::2], q) == INVALID           # elements apart
    assert rope_code(rows(4, 5).transpose(0, 1), q) == INVALID          # heads not side by side
    assert rope_code(None, q, k, k) == INVALID                          # an output without its input
    assert code_of(gdn.gdn_rope, gdn.make_attn_dims(4, 2, 64, 16),
                   gdn.make_rope(64, torch.ones(32), i32(5)), None, None) == INVALID


def append_args(**kw):
    a = dict(dims=gdn.make_attn_dims(4, 2, 64, 16),
             batch=gdn.make_kv_batch(2, 5, 4, 3, i32(2), i32(2), i32(2), i32(2, 2)),
             rope=gdn.make_rope(64, torch.ones(32), i32(5)), q=rows(5, 4), k=rows(5, 2),
             v=rows(5, 2), q_out=rows(5, 4), k_cache=torch.zeros(3, 2, 16, 64, dtype=BF),
             v_cache=torch.zeros(3, 2, 16, 64, dtype=BF), status=i32(1))
    a.update(kw)
    return a


def attn_args(**kw):
    a = append_args()
    for name in ("rope", "q_out", "k", "v"):
        del a[name]
    n = [size(a["dims"], a["batch"]) for size in
         (gdn.gdn_attn_plan_bytes, gdn.gdn_attn_workspace_bytes)]
    a.update(plan=torch.zeros(n[0], dtype=torch.uint8), o=rows(5, 4), lse=torch.zeros(5, 4),
             workspace=torch.zeros(n[1], dtype=torch.uint8), workspace_bytes=n[1])
    a.update(kw)
    return a


@pytest.mark.skipif(torch.cuda.is_available(), reason="host memory is passed on to the launch")
def test_calls_that_fit_reach_the_launch():
    assert code_of(gdn.gdn_kv_append, **append_args()) != INVALID
    assert code_of(gdn.gdn_kv_append, **append_args(k=rows(8, 2), q_out=rows(6, 4))) != INVALID
    assert code_of(gdn.gdn_attn, **attn_args()) != INVALID


@pytest.mark.parametrize("name,heads", [("q", 4), ("k", 2), ("v", 2), ("q_out", 4)])
def test_append_rows_that_do_not_fit_are_refused(name, heads):
    for t in (rows(4, heads), rows(5, heads - 1), rows(5, heads, 128), rows(5, heads, dtype=HF),
              rows(heads, 5).transpose(0, 1)):
        assert code_of(gdn.gdn_kv_append, **append_args(**{name: t})) == INVALID, t.shape


def test_attn_query_rows_that_do_not_fit_are_refused():
    for t in (rows(4, 4), rows(5, 3), rows(5, 4, 128), rows(5, 4, dtype=HF)):
        assert code_of(gdn.gdn_attn, **attn_args(q=t)) == INVALID, t.shape


def refused(make, *args, **kw):
    with pytest.raises(gdn.GdnError) as e:
        make(*args, **kw)
    return e.value.code == INVALID


def test_index_tensors_that_are_not_int32_are_refused():
    """torch counts in int64 unless told otherwise; read as int32 every other number is 0."""
    freq = torch.ones(32)
    assert refused(gdn.make_rope, 64, freq, torch.arange(5))
    assert refused(gdn.make_rope, 64, freq, i32(5), axis=torch.zeros(32, dtype=torch.int64))
    assert refused(gdn.make_rope, 64, freq.double(), i32(5))
    assert refused(gdn.make_rope, 64, freq.bfloat16(), i32(5))
    good = [i32(2), i32(2), i32(2), i32(2, 3), i32(1), i32(1), i32(1)]
    gdn.make_kv_batch(2, 5, 4, 9, *good)
    for i, t in enumerate(good):
        bad = list(good)
        bad[i] = t.long()
        assert refused(gdn.make_kv_batch, 2, 5, 4, 9, *bad), i


def test_index_tensors_that_are_short_or_strided_are_refused():
    freq = torch.ones(32)
    assert refused(gdn.make_rope, 64, torch.ones(31), i32(5))
    assert refused(gdn.make_rope, 64, torch.ones(64)[::2], i32(5))
    assert refused(gdn.make_rope, 64, freq, i32(5), axis=i32(31))
    assert refused(gdn.make_rope, 64, freq, i32(3, 8)[:, :5])      # three axes cut from longer ones
    assert refused(gdn.make_rope, 64, freq, i32(5, 3).t())
    good = [i32(4), i32(4), i32(4), i32(4, 3), i32(2), i32(2), i32(2)]
    gdn.make_kv_batch(4, 5, 4, 9, *good)
    for i, t in enumerate(good):
        if i != 4:                                                 # (the groups are as many as it holds)
            bad = list(good)
            bad[i] = t[:-1]
            assert refused(gdn.make_kv_batch, 4, 5, 4, 9, *bad), i
        bad = list(good)
        bad[i] = torch.stack([t, t], -1)[..., 0] if t.dim() == 1 else i32(4, 8)[:, :3]
        assert refused(gdn.make_kv_batch, 4, 5, 4, 9, *bad), i
    assert refused(gdn.make_kv_batch, 4, 5, 4, 9, *good[:3], i32(3, 4).t())


def test_positions_for_other_rows_are_refused():
    q = rows(5, 4)
    assert rope_code(q, q, positions=i32(4)) == INVALID
    assert rope_code(q, q, positions=i32(3, 6)) == INVALID         # each axis would start elsewhere
    assert rope_code(q, q, positions=i32(3, 4)) == INVALID
    for n in (4, 3):
        short = gdn.make_rope(64, torch.ones(32), i32(n))
        assert code_of(gdn.gdn_kv_append, **append_args(rope=short)) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="host memory is passed on to the launch")
def test_positions_with_room_reach_the_launch():
    q = rows(5, 4)
    assert rope_code(q, q, positions=i32(9)) != INVALID            # one axis: the first ones
    assert rope_code(q, q, positions=i32(3, 5)) != INVALID
    none = gdn.make_rope(0, None, None)
    assert code_of(gdn.gdn_rope, gdn.make_attn_dims(4, 2, 64, 16), none, q, q) != INVALID


def not_fitting(t, other):
    """Tensors that hold other elements than a dense t does: too few, strided, of another type."""
    wide = torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype)
    return [t[:-1], wide[..., ::2], wide[..., :t.shape[-1]], t.to(other),
            torch.zeros_like(t).transpose(0, 1)]


@pytest.mark.parametrize("name", ["k_cache", "v_cache"])
def test_caches_that_are_not_dense_are_refused(name):
    for t in not_fitting(torch.zeros(3, 2, 16, 64, dtype=BF), HF):
        assert code_of(gdn.gdn_kv_append, **append_args(**{name: t})) == INVALID, t.shape
        assert code_of(gdn.gdn_attn, **attn_args(**{name: t})) == INVALID, t.shape


def test_outputs_that_are_not_dense_are_refused():
    for t in not_fitting(rows(5, 4), HF):
        assert code_of(gdn.gdn_attn, **attn_args(o=t)) == INVALID, t.shape
    for t in not_fitting(torch.zeros(5, 4), torch.float64):
        assert code_of(gdn.gdn_attn, **attn_args(lse=t)) == INVALID, t.shape


@pytest.mark.skipif(torch.cuda.is_available(), reason="host memory is passed on to the launch")
def test_outputs_and_caches_of_other_shapes_reach_the_launch():
    assert code_of(gdn.gdn_attn, **attn_args(o=torch.zeros(5, 256, dtype=BF), lse=None)) != INVALID
    assert code_of(gdn.gdn_attn, **attn_args(o=rows(9, 4))) != INVALID
    big = torch.zeros(8, 2, 16, 64, dtype=BF)
    assert code_of(gdn.gdn_attn, **attn_args(k_cache=big, v_cache=big)) != INVALID


def test_abi_version_tells_the_attention_layer_calls():
    assert gdn.gdn_abi_version() >= (2 << 16 | 2)
