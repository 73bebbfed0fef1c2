"""Host-side checks of the attention-layer calls that need no GPU: bad
arguments are refused before anything is launched, sizes are as declared."""
import ctypes
import os
import shutil
import subprocess

import pytest

import gated_deltanet_linear_14_gb300 as gdn
from gated_deltanet_linear_14_gb300 import build as gbuild

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -4


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gdn.load_library()


def dims(**kw):
    d = gdn.make_attn_dims(32, 8, 128, 64)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def batch(**kw):
    b = gdn.KvBatch(4, 4, 1, 9, 3, 0, 16, 16, 16, 16, None, None, None)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def rope(**kw):
    r = gdn.RopeParams(64, 1, 0, 16, None, 16)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


R = ctypes.byref


def call_rope(lib, d=None, r=None, rows=4, q=16, qs=4096, qo=32, qos=4096, k=None, ks=0, ko=None,
              kos=0, inverse=0):
    d, r = d or dims(), r or rope()
    return lib.gdn_rope(R(d), R(r), rows, q, qs, qo, qos, k, ks, ko, kos, inverse, None)


def call_append(lib, d=None, b=None, r=None, q=16, qs=4096, k=16, ks=1024, v=16, vs=1024, qo=32,
                qos=4096, kc=16, vc=16, status=16):
    d, b, r = d or dims(), b or batch(), r or rope()
    return lib.gdn_kv_append(R(d), R(b), R(r), q, qs, k, ks, v, vs, qo, qos, kc, vc, status, None)


def call_attn(lib, d=None, b=None, plan=16, q=16, qs=4096, kc=16, vc=16, o=16, ws=16, n=1 << 40,
              status=16):
    d, b = d or dims(), b or batch()
    return lib.gdn_attn(R(d), R(b), plan, q, qs, kc, vc, o, None, ws, n, status, None)


def call_plan(lib, d=None, b=None, plan=16, n=1 << 40, status=16):
    d, b = d or dims(), b or batch()
    return lib.gdn_attn_plan(R(d), R(b), plan, n, status, None)


BAD_DIMS = [("num_q_heads", 0, INVALID), ("num_kv_heads", -1, INVALID), ("head_dim", 0, INVALID),
            ("io_dtype", 3, INVALID), ("scale", float("nan"), INVALID),
            ("num_kv_heads", 5, UNSUPPORTED)]


@pytest.mark.parametrize("field,value,code", BAD_DIMS)
def test_dims_refused_everywhere(lib, field, value, code):
    d = dims(**{field: value})
    assert call_rope(lib, d=d) == code
    assert call_append(lib, d=d) == code
    assert call_attn(lib, d=d) == code
    assert call_plan(lib, d=d) == code
    assert lib.gdn_attn_plan_bytes(R(d), R(batch())) == 0
    assert lib.gdn_attn_workspace_bytes(R(d), R(batch())) == 0


@pytest.mark.parametrize("field,value,code", [
    ("head_dim", 96, UNSUPPORTED), ("page_size", 8, UNSUPPORTED), ("page_size", 48, UNSUPPORTED),
    ("page_size", 512, UNSUPPORTED), ("page_size", 0, INVALID), ("io_dtype", gdn.GDN_F32, UNSUPPORTED)])
def test_cache_dims_refused(lib, field, value, code):
    d = dims(**{field: value})
    assert call_append(lib, d=d) == code
    assert call_attn(lib, d=d) == code
    assert call_plan(lib, d=d) == code


def test_too_many_queries_per_key_head(lib):
    d = gdn.make_attn_dims(258, 2, 128, 64)
    assert call_attn(lib, d=d, qs=258 * 128) == UNSUPPORTED
    assert call_plan(lib, d=d) == UNSUPPORTED


@pytest.mark.parametrize("field,value,code", [
    ("num_requests", -1, INVALID), ("num_rows", -1, INVALID), ("max_rows", -1, INVALID),
    ("num_pages", -1, INVALID), ("max_pages", -1, INVALID), ("num_groups", -1, INVALID),
    ("num_requests", 70000, UNSUPPORTED), ("row_start", None, INVALID), ("row_len", None, INVALID),
    ("kv_len", None, INVALID), ("page_table", None, INVALID)])
def test_batch_refused(lib, field, value, code):
    b = batch(**{field: value})
    assert call_append(lib, b=b) == code
    assert call_attn(lib, b=b) == code
    assert call_plan(lib, b=b) == code


def test_groups_refused(lib):
    assert call_plan(lib, b=batch(num_groups=5)) == UNSUPPORTED   # more groups than requests
    assert call_plan(lib, b=batch(num_groups=2)) == INVALID       # no group arrays
    assert call_attn(lib, b=batch(num_groups=2, group_start=16, group_len=16)) == INVALID


@pytest.mark.parametrize("field,value", [
    ("rotary_dim", -2), ("rotary_dim", 63), ("rotary_dim", 130), ("num_axes", 0),
    ("interleaved", 2), ("inv_freq", None), ("positions", None)])
def test_rope_params_refused(lib, field, value):
    r = rope(**{field: value})
    assert call_rope(lib, r=r) == INVALID
    assert call_append(lib, r=r) == INVALID


def test_rope_buffers_refused(lib):
    assert call_rope(lib, rows=-1) == INVALID
    assert call_rope(lib, inverse=2) == INVALID
    assert call_rope(lib, qo=None) == INVALID
    assert call_rope(lib, q=None) == INVALID                       # an output without its input
    assert call_rope(lib, q=None, qo=None) == INVALID              # nothing to rotate
    assert call_rope(lib, qs=4095) == INVALID                      # rows overlap
    assert call_rope(lib, qos=-4096) == INVALID
    assert call_rope(lib, q=32, qs=8192) == INVALID                # in place with two strides
    assert call_rope(lib, d=dims(head_dim=2048)) == UNSUPPORTED
    assert call_rope(lib, d=dims(head_dim=127), r=rope(rotary_dim=126)) == UNSUPPORTED
    assert call_rope(lib, rows=0, q=None, qo=None) == OK           # nothing to do


def test_append_buffers_refused(lib):
    for name in ("k", "v", "kc", "vc", "status", "qo"):
        assert call_append(lib, **{name: None}) == INVALID
    assert call_append(lib, ks=1023) == INVALID
    assert call_append(lib, vs=0) == INVALID
    d, b = dims(), batch()
    assert lib.gdn_kv_append(R(d), R(b), None, 16, 4096, 16, 1024, 16, 1024, 32, 4096, 16, 16, 16,
                             None) == INVALID                      # q without a rotation
    assert call_append(lib, b=batch(num_requests=0)) == OK


def test_attn_buffers_refused(lib):
    for name in ("plan", "q", "kc", "vc", "o", "ws", "status"):
        assert call_attn(lib, **{name: None}) == INVALID
    assert call_attn(lib, plan=24) == INVALID
    assert call_attn(lib, ws=8) == INVALID
    assert call_attn(lib, qs=4095) == INVALID
    assert call_attn(lib, qs=4100) == UNSUPPORTED
    assert call_attn(lib, q=18) == UNSUPPORTED
    assert call_attn(lib, o=8) == UNSUPPORTED
    assert call_attn(lib, kc=8) == UNSUPPORTED
    need = lib.gdn_attn_workspace_bytes(R(dims()), R(batch()))
    assert need > 0 and call_attn(lib, n=need - 1) == WORKSPACE
    assert call_attn(lib, b=batch(num_requests=0)) == OK


def test_plan_buffers_refused(lib):
    assert call_plan(lib, plan=None) == INVALID
    assert call_plan(lib, status=None) == INVALID
    assert call_plan(lib, plan=24) == INVALID
    need = lib.gdn_attn_plan_bytes(R(dims()), R(batch()))
    assert need > 0 and call_plan(lib, n=need - 1) == WORKSPACE


def test_structs_match_the_header(tmp_path):
    """A C client sees the binding's sizes and offsets."""
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    pairs = [(gdn.AttnDims, "gdn_attn_dims"), (gdn.RopeParams, "gdn_rope_params"),
             (gdn.KvBatch, "gdn_kv_batch")]
    lines, want = [], []
    for cls, name in pairs:
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(cls))
        for field, _ in cls._fields_:
            lines.append(f'printf("%zu\\n", offsetof({name}, {field}));')
            want.append(getattr(cls, field).offset)
    lines.append('printf("%d\\n", GDN_F16);')
    want.append(gdn.GDN_F16)
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "gdn.h"\nint main(void) {\n'
                   + "\n".join(lines) + "\nreturn 0; }\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = tmp_path / "sizes"
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(root, "include"),
                    str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True,
                                          text=True).stdout.split()]
    assert got == want
