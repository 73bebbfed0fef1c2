"""Checks of the norms' and the 8-bit cache's calls that need no GPU: what does not fit is refused
before anything is launched, sizes are as declared."""
import ctypes
import gc
import os
import shutil
import subprocess
import weakref

import pytest
import torch

import gated_deltanet_linear_14_gb300 as gdn
from gated_deltanet_linear_14_gb300 import build as gbuild
from gated_deltanet_linear_14_gb300.pages import Kv8Cache

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -4
R = ctypes.byref
BF, HF, F32, E4 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def lib():
    gbuild.build()
    return gdn.load_library()


def made(cls, *fields, **kw):
    s = cls(*fields)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def dims(**kw):
    return made(gdn.AttnDims, 32, 8, 128, 64, gdn.GDN_BF16, 0.0, **kw)


def batch(**kw):
    return made(gdn.KvBatch, 4, 4, 1, 9, 3, 0, 16, 16, 16, 16, None, None, None, **kw)


def rope(**kw):
    return made(gdn.RopeParams, 64, 1, 0, 16, None, 16, **kw)


def norm(**kw):
    return made(gdn.HeadNorm, 16, 16, 1e-6, 0.0, **kw)


def cache(**kw):
    return made(gdn.Kv8Codes, 16, 16, 16, 16, **kw)


def call_norm(lib, d=None, n=None, r=None, rows=4, q=16, qs=4096, qo=32, qos=4096, k=None, ks=0,
              ko=None, kos=0):
    return lib.gdn_norm_rope(R(d or dims()), R(n or norm()), R(r or rope()), rows, q, qs, qo, qos, k,
                             ks, ko, kos, None)


def call_append(lib, d=None, b=None, n=None, r=None, q=16, qs=4096, k=16, ks=1024, v=16, vs=1024,
                qo=32, qos=4096, c=None, status=16):
    return lib.gdn_kv8_append(R(d or dims()), R(b or batch()), R(n or norm()), R(r or rope()), q, qs,
                              k, ks, v, vs, qo, qos, R(c or cache()), status, None)


def call_read(lib, d=None, b=None, c=None, k=16, ks=1024, v=16, vs=1024, status=16):
    return lib.gdn_kv8_read(R(d or dims()), R(b or batch()), R(c or cache()), k, ks, v, vs, status,
                            None)


def call_plan(lib, d=None, b=None, plan=16, n=1 << 40, status=16):
    return lib.gdn_kv8_attn_plan(R(d or dims()), R(b or batch()), plan, n, status, None)


def call_attn(lib, d=None, b=None, plan=16, q=16, qs=4096, c=None, o=16, ws=16, n=1 << 40,
              status=16):
    return lib.gdn_kv8_attn(R(d or dims()), R(b or batch()), plan, q, qs, R(c or cache()), o, None,
                            ws, n, status, None)


@pytest.mark.parametrize("field,value,code", [
    ("num_q_heads", 0, INVALID), ("num_kv_heads", -1, INVALID), ("head_dim", 0, INVALID),
    ("io_dtype", 3, INVALID), ("scale", float("nan"), INVALID), ("num_kv_heads", 5, UNSUPPORTED)])
def test_dims_refused_everywhere(lib, field, value, code):
    d = dims(**{field: value})
    for call in (call_norm, call_append, call_read, call_plan, call_attn):
        assert call(lib, d=d) == code, call
    assert lib.gdn_kv8_attn_plan_bytes(R(d), R(batch())) == 0
    assert lib.gdn_kv8_attn_workspace_bytes(R(d), R(batch())) == 0


@pytest.mark.parametrize("field,value,code", [
    ("head_dim", 96, UNSUPPORTED), ("page_size", 8, UNSUPPORTED), ("page_size", 48, UNSUPPORTED),
    ("page_size", 512, UNSUPPORTED), ("page_size", 0, INVALID)])
def test_cache_dims_refused(lib, field, value, code):
    d = dims(**{field: value})
    for call in (call_append, call_read, call_plan, call_attn):
        assert call(lib, d=d) == code, call


def test_types_refused(lib):
    d = dims(io_dtype=gdn.GDN_F32)
    for call in (call_append, call_plan, call_attn):
        assert call(lib, d=d) == UNSUPPORTED
    d = gdn.make_attn_dims(258, 2, 128, 64)
    assert call_attn(lib, d=d, qs=258 * 128) == UNSUPPORTED and call_plan(lib, d=d) == UNSUPPORTED


@pytest.mark.parametrize("field,value,code", [
    ("num_requests", -1, INVALID), ("num_rows", -1, INVALID), ("max_rows", -1, INVALID),
    ("num_pages", -1, INVALID), ("max_pages", -1, INVALID), ("num_groups", -1, INVALID),
    ("num_requests", 70000, UNSUPPORTED), ("row_start", None, INVALID), ("row_len", None, INVALID),
    ("kv_len", None, INVALID), ("page_table", None, INVALID)])
def test_batch_refused(lib, field, value, code):
    b = batch(**{field: value})
    for call in (call_append, call_read, call_plan, call_attn):
        assert call(lib, b=b) == code, call


@pytest.mark.parametrize("field,value", [("eps", -1e-6), ("eps", float("nan")),
                                          ("eps", float("inf")), ("offset", float("nan")),
                                          ("offset", float("-inf"))])
def test_norm_refused(lib, field, value):
    assert call_norm(lib, n=norm(**{field: value})) == INVALID
    assert call_append(lib, n=norm(**{field: value})) == INVALID


@pytest.mark.parametrize("field,value", [
    ("rotary_dim", -2), ("rotary_dim", 63), ("rotary_dim", 130), ("num_axes", 0),
    ("interleaved", 2), ("inv_freq", None), ("positions", None)])
def test_rope_params_refused(lib, field, value):
    assert call_norm(lib, r=rope(**{field: value})) == INVALID
    assert call_append(lib, r=rope(**{field: value})) == INVALID


def test_norm_buffers_refused(lib):
    assert call_norm(lib, rows=-1) == INVALID
    assert call_norm(lib, qo=None) == INVALID and call_norm(lib, q=None) == INVALID
    assert call_norm(lib, q=None, qo=None) == INVALID              # nothing to norm
    assert call_norm(lib, qs=4095) == INVALID and call_norm(lib, qos=-4096) == INVALID
    assert call_norm(lib, q=32, qs=8192) == INVALID                # in place with two strides
    assert call_norm(lib, k=16, ks=1023, ko=16, kos=1024) == INVALID
    assert call_norm(lib, d=dims(head_dim=2048)) == UNSUPPORTED
    assert call_norm(lib, d=dims(head_dim=127), r=rope(rotary_dim=126)) == UNSUPPORTED
    assert call_norm(lib, rows=0, q=None, qo=None) == OK           # nothing to do
    assert lib.gdn_norm_rope(R(dims()), None, R(rope()), 4, 16, 4096, 32, 4096, None, 0, None, 0,
                             None) == INVALID


def test_append_buffers_refused(lib):
    for name in ("k", "v", "qo", "status"):
        assert call_append(lib, **{name: None}) == INVALID
    for name in ("k", "v", "k_exp", "v_exp"):
        assert call_append(lib, c=cache(**{name: None})) == INVALID
    assert call_append(lib, c=cache(v=24)) == UNSUPPORTED
    assert call_append(lib, ks=1023) == INVALID and call_append(lib, vs=0) == INVALID
    for kw in (dict(q=18), dict(k=24), dict(qo=40), dict(qs=4100), dict(vs=1028),
               dict(r=rope(rotary_dim=40))):
        assert call_append(lib, **kw) == UNSUPPORTED, kw
    d, b, c = dims(), batch(), cache()
    bare = lambda q, qo: lib.gdn_kv8_append(R(d), R(b), None, None, q, 4096, 16, 1024, 16, 1024,  # noqa: E731
                                            qo, 4096, R(c), 16, None)
    assert bare(16, 32) == INVALID                                 # nothing to do to the queries
    assert lib.gdn_kv8_append(R(d), R(b), None, None, None, 0, 16, 1024, 16, 1024, None, 0, None, 16,
                              None) == INVALID                     # no cache
    assert call_append(lib, b=batch(num_requests=0)) == OK


def test_read_buffers_refused(lib):
    assert call_read(lib, k=None, v=None) == INVALID and call_read(lib, status=None) == INVALID
    assert call_read(lib, ks=1000) == INVALID
    assert call_read(lib, c=cache(k=None)) == INVALID and call_read(lib, c=cache(v=8)) == UNSUPPORTED
    assert call_read(lib, b=batch(max_rows=0)) == OK


def test_attn_buffers_refused(lib):
    for name in ("plan", "q", "o", "ws", "status"):
        assert call_attn(lib, **{name: None}) == INVALID
    assert call_attn(lib, plan=24) == INVALID and call_attn(lib, ws=8) == INVALID
    assert call_attn(lib, qs=4095) == INVALID
    assert call_attn(lib, qs=4100) == UNSUPPORTED and call_attn(lib, q=18) == UNSUPPORTED
    assert call_attn(lib, o=8) == UNSUPPORTED and call_attn(lib, c=cache(k=8)) == UNSUPPORTED
    assert call_attn(lib, c=cache(v_exp=None)) == INVALID
    need = lib.gdn_kv8_attn_workspace_bytes(R(dims()), R(batch()))
    assert need > 0 and call_attn(lib, n=need - 1) == WORKSPACE
    need = lib.gdn_kv8_attn_plan_bytes(R(dims()), R(batch()))
    assert need > 0 and call_plan(lib, n=need - 1) == WORKSPACE
    assert call_plan(lib, plan=None) == INVALID and call_plan(lib, plan=24) == INVALID
    assert call_plan(lib, b=batch(num_groups=5)) == UNSUPPORTED
    assert call_attn(lib, b=batch(num_groups=2, group_start=16, group_len=16)) == INVALID
    assert call_attn(lib, b=batch(num_requests=0)) == OK


def test_copies_are_for_steps_of_many_rows_a_request(lib):
    """By the rows that the requests can have, not by the size of the row buffers."""
    def sizes(n, rows, most):
        d, b = dims(), batch(num_requests=n, num_rows=rows, max_rows=most, max_pages=100)
        return [size(R(d), R(b))
                for size in (lib.gdn_attn_workspace_bytes, lib.gdn_kv8_attn_workspace_bytes)]

    for n, rows, most in ((1, 4096, 1), (4, 4096, 8), (1, 1 << 20, 255), (8, 1 << 20, 255)):
        plain, codes8 = sizes(n, rows, most)
        assert plain == codes8 > 0, (n, rows, most)
    for n, rows, most in ((1, 256, 256), (8, 2048, 2048), (8, 1 << 20, 256)):
        plain, codes8 = sizes(n, rows, most)
        assert codes8 > plain + 2 * n * 100 * 2 * 8 * 64 * 128 - 1, (n, rows, most)


def test_a_workspace_without_room_for_copies_is_taken(lib):
    d, b = dims(), batch(num_requests=1, num_rows=2048, max_rows=2048, max_pages=100)
    least = lib.gdn_attn_workspace_bytes(R(d), R(b))
    assert least < lib.gdn_kv8_attn_workspace_bytes(R(d), R(b))
    assert call_attn(lib, b=b, n=least - 1) == WORKSPACE
    if not torch.cuda.is_available():   # (host memory is passed on to the launch)
        assert call_attn(lib, b=b, n=least) not in (WORKSPACE, INVALID, UNSUPPORTED)


def test_structs_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    lines, want = ['printf("%d\\n", GDN_KV8_BLOCK);'], [16]
    for cls, name in ((gdn.HeadNorm, "gdn_head_norm"), (gdn.Kv8Codes, "gdn_kv8_cache")):
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(cls))
        for field, _ in cls._fields_:
            lines.append(f'printf("%zu\\n", offsetof({name}, {field}));')
            want.append(getattr(cls, field).offset)
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "gdn.h"\nint main(void) {\n'
                   + "\n".join(lines) + "\nreturn 0; }\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = tmp_path / "sizes"
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(root, "include"),
                    str(src), "-o", str(exe)], check=True)
    assert [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True,
                                           text=True).stdout.split()] == want


def test_abi_version_tells_the_8_bit_calls():
    assert gdn.gdn_abi_version() >= (2 << 16 | 3)


# ------------------------------------------------------------------ binding

def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def rows(n, heads, dim=64, dtype=BF):
    return torch.zeros(n, heads, dim, dtype=dtype)


def code_of(call, *args, **kw):
    with pytest.raises(gdn.GdnError) as e:
        call(*args, stream=0, **kw)
    return e.value.code


def small(**kw):
    d = gdn.make_attn_dims(4, 2, 64, 16)
    a = dict(dims=d, batch=gdn.make_kv_batch(2, 5, 4, 3, i32(2), i32(2), i32(2), i32(2, 2)),
             norm=gdn.make_head_norm(torch.ones(64), torch.ones(64)),
             rope=gdn.make_rope(64, torch.ones(32), i32(5)), q=rows(5, 4), k=rows(5, 2),
             v=rows(5, 2), q_out=rows(5, 4), cache=Kv8Cache(d, 3, device="cpu").codes, status=i32(1))
    a.update(kw)
    return a


def read_args(**kw):
    a = small()
    return {**{x: a[x] for x in ("dims", "batch", "cache", "status")}, "k_out": rows(5, 2),
            "v_out": rows(5, 2), **kw}


def attn_args(**kw):
    a = small()
    n = [size(a["dims"], a["batch"]) for size in
         (gdn.gdn_kv8_attn_plan_bytes, gdn.gdn_kv8_attn_workspace_bytes)]
    return {**{x: a[x] for x in ("dims", "batch", "q", "cache", "status")},
            "plan": torch.zeros(n[0], dtype=torch.uint8), "o": rows(5, 4), "lse": torch.zeros(5, 4),
            "workspace": torch.zeros(n[1], dtype=torch.uint8), "workspace_bytes": n[1], **kw}


@pytest.mark.skipif(torch.cuda.is_available(), reason="host memory is passed on to the launch")
def test_calls_that_fit_reach_the_launch():
    assert code_of(gdn.gdn_kv8_append, **small()) != INVALID
    assert code_of(gdn.gdn_kv8_read, **read_args()) != INVALID
    assert code_of(gdn.gdn_kv8_attn, **attn_args()) != INVALID


def test_rows_that_do_not_fit_are_refused():
    for name, heads in (("q", 4), ("k", 2), ("v", 2), ("q_out", 4)):
        for t in (rows(4, heads), rows(5, heads - 1), rows(5, heads, 128),
                  rows(5, heads, dtype=HF), rows(heads, 5).transpose(0, 1)):
            assert code_of(gdn.gdn_kv8_append, **small(**{name: t})) == INVALID, (name, t.shape)
    for name in ("k_out", "v_out"):
        for t in (rows(4, 2), rows(5, 1), rows(5, 2, 128), rows(5, 2, dtype=F32)):
            assert code_of(gdn.gdn_kv8_read, **read_args(**{name: t})) == INVALID, (name, t.shape)
    for name, t in (("q", rows(4, 4)), ("o", rows(4, 4)), ("o", rows(5, 4, dtype=HF)),
                    ("lse", torch.zeros(4, 4)), ("lse", torch.zeros(5, 4, dtype=torch.float64))):
        assert code_of(gdn.gdn_kv8_attn, **attn_args(**{name: t})) == INVALID, (name, t.shape)
    d, n, r = gdn.make_attn_dims(4, 2, 64, 16), gdn.make_head_norm(), gdn.make_rope(64, torch.ones(32), i32(5))
    for q, out in ((rows(5, 4), rows(4, 4)), (rows(5, 3), rows(5, 4)), (rows(5, 4, dtype=HF), rows(5, 4)),
                   (rows(6, 4), rows(5, 4))):
        assert code_of(gdn.gdn_norm_rope, d, n, r, q, out) == INVALID
    assert code_of(gdn.gdn_norm_rope, d, n, r, None, None) == INVALID
    assert code_of(gdn.gdn_norm_rope, d, gdn.make_head_norm(torch.ones(32)), r, rows(5, 4), rows(5, 4)) == INVALID


def test_caches_that_do_not_fit_are_refused():
    def cache_of(k, e):
        return gdn.make_kv8_cache(k, k, e, e)

    k, e = torch.zeros(3, 2, 16, 64).to(E4), torch.zeros(3, 2, 1, dtype=torch.int8)
    good = cache_of(k, e)
    assert good.k == k.data_ptr() and good.v_exp == e.data_ptr()
    cache_of(k.view(torch.uint8), e)
    for bad in ((k.float(), e), (k, e.int()), (k, None), (k, e[:2]), (k[..., ::2], e),
                (k.view(torch.uint8).transpose(1, 2), e), (k[0], e)):
        with pytest.raises(gdn.GdnError):
            cache_of(*bad)
    with pytest.raises(gdn.GdnError):
        gdn.make_kv8_cache(k, torch.zeros(4, 2, 16, 64).to(E4), e, torch.zeros(4, 2, 1, dtype=torch.int8))
    other = cache_of(torch.zeros(3, 2, 32, 64).to(E4), torch.zeros(3, 2, 2, dtype=torch.int8))
    few = cache_of(k[:2], e[:2])
    for c in (other, few, None):
        assert code_of(gdn.gdn_kv8_append, **small(cache=c)) == INVALID
        assert code_of(gdn.gdn_kv8_read, **read_args(cache=c)) == INVALID
        assert code_of(gdn.gdn_kv8_attn, **attn_args(cache=c)) == INVALID


def test_weights_that_do_not_fit_are_refused():
    for w in (torch.ones(64, dtype=BF), torch.ones(64, dtype=torch.float64), torch.ones(128)[::2]):
        for kw in (dict(q_weight=w), dict(k_weight=w)):
            with pytest.raises(gdn.GdnError):
                gdn.make_head_norm(**kw)
    short = gdn.make_head_norm(torch.ones(64), torch.ones(63))
    assert code_of(gdn.gdn_kv8_append, **small(norm=short)) == INVALID


def test_structures_keep_their_tensors():
    for make, args in ((gdn.make_head_norm, lambda: [torch.ones(64), torch.ones(64)]),
                       (gdn.make_kv8_cache, lambda: [torch.zeros(1, 1, 16, 64).to(E4) for _ in range(2)]
                        + [torch.zeros(1, 1, 1, dtype=torch.int8) for _ in range(2)])):
        tensors = args()
        refs = [weakref.ref(t) for t in tensors]
        s = make(*tensors)
        del tensors
        gc.collect()
        assert all(r() is not None for r in refs)
        del s
        gc.collect()
        assert all(r() is None for r in refs)
