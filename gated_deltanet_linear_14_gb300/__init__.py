"""Python binding of libgdn.so, the GB300 Gated DeltaNet layer core.

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in ``include/gdn.h``. PyTorch provides
device memory and streams. The binding raises if the library is missing; it
never falls back to another implementation.

Entry points (same names as the C ABI): ``gdn_conv``, ``gdn_seq``,
``gdn_decode``, ``gdn_prefill``, ``gdn_spec_verify``, ``gdn_spec_step``, ``gdn_spec_slots``,
``gdn_chunk_prefill``, ``gdn_chunk_prefill_noalloc``, ``gdn_page_to_slots``, ``gdn_slots_to_page``,
``gdn_chunk_prefill_workspace_bytes``, ``gdn_page_layout``,
``gdn_slot_layout``, ``gdn_check_bounded_wait``, ``gdn_strerror``,
``gdn_abi_version``; for the attention layers between GDN layers ``gdn_rope``,
``gdn_kv_append``, ``gdn_attn_plan``, ``gdn_attn``, ``gdn_attn_plan_bytes``,
``gdn_attn_workspace_bytes``; norms of queries and keys and an 8-bit cache for them
``gdn_norm_rope``, ``gdn_kv8_append``, ``gdn_kv8_read``, ``gdn_kv8_attn_plan``,
``gdn_kv8_attn``, ``gdn_kv8_attn_plan_bytes``, ``gdn_kv8_attn_workspace_bytes``.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libgdn.so")

GDN_F32 = 0
GDN_BF16 = 1
GDN_F16 = 2
GDN_REQ_FRESH = 0x1
GDN_REQ_SPEC = 0x2
GDN_REQ_PARITY = 0x4

STATUS = {
    0: "GDN_OK", -1: "GDN_ERR_INVALID_ARG", -2: "GDN_ERR_UNSUPPORTED", -3: "GDN_ERR_LAUNCH",
    -4: "GDN_ERR_WORKSPACE", -5: "GDN_ERR_NO_DEVICE", 1: "GDN_DEV_BAD_PAGE",
    2: "GDN_DEV_BAD_ROWS", 3: "GDN_DEV_BAD_ACCEPTED", 4: "GDN_DEV_STALE_STEP",
    5: "GDN_DEV_TOO_MANY_CANDIDATES", 6: "GDN_DEV_RECORD_OPEN", 7: "GDN_DEV_BAD_FLAG",
    8: "GDN_DEV_TIMEOUT",
}
CODES = {v: k for k, v in STATUS.items()}


class GdnError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        super().__init__(f"{where}: {STATUS.get(code, code)} ({gdn_strerror(code)})")


class Dims(ctypes.Structure):
    _fields_ = [("num_k_heads", ctypes.c_int32), ("num_v_heads", ctypes.c_int32),
                ("head_k_dim", ctypes.c_int32), ("head_v_dim", ctypes.c_int32),
                ("conv_width", ctypes.c_int32), ("max_candidates", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("state_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32)]

    @property
    def C(self):
        return 2 * self.num_k_heads * self.head_k_dim + self.num_v_heads * self.head_v_dim


class Params(ctypes.Structure):
    _fields_ = [("A_log", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p),
                ("conv_bias", ctypes.c_void_p), ("scale", ctypes.c_float),
                ("norm_eps", ctypes.c_float), ("gate_mode", ctypes.c_int32)]


class Batch(ctypes.Structure):
    _fields_ = [("num_requests", ctypes.c_int32), ("num_rows", ctypes.c_int32),
                ("max_rows", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("row_start", ctypes.c_void_p), ("row_len", ctypes.c_void_p),
                ("page", ctypes.c_void_p), ("flags", ctypes.c_void_p),
                ("n_accepted", ctypes.c_void_p), ("order", ctypes.c_void_p)]


class PageLayout(ctypes.Structure):
    _fields_ = [("page_bytes", ctypes.c_size_t), ("window_offset", ctypes.c_size_t),
                ("window_bytes", ctypes.c_size_t), ("state_offset", ctypes.c_size_t),
                ("state_bytes", ctypes.c_size_t), ("record_offset", ctypes.c_size_t),
                ("record_bytes", ctypes.c_size_t), ("flag_offset", ctypes.c_size_t)]


class SlotLayout(ctypes.Structure):
    _fields_ = [("pool_bytes", ctypes.c_size_t), ("slot_bytes", ctypes.c_size_t),
                ("state_offset", ctypes.c_size_t), ("window_offset", ctypes.c_size_t)]


class AttnDims(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


class RopeParams(ctypes.Structure):
    columns = None  # of the positions, where make_rope saw them
    _fields_ = [("rotary_dim", ctypes.c_int32), ("num_axes", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("inv_freq", ctypes.c_void_p),
                ("axis", ctypes.c_void_p), ("positions", ctypes.c_void_p)]


class KvBatch(ctypes.Structure):
    _fields_ = [("num_requests", ctypes.c_int32), ("num_rows", ctypes.c_int32),
                ("max_rows", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("num_groups", ctypes.c_int32),
                ("row_start", ctypes.c_void_p), ("row_len", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("group_start", ctypes.c_void_p), ("group_len", ctypes.c_void_p),
                ("group_pages", ctypes.c_void_p)]


class HeadNorm(ctypes.Structure):
    width = None  # of the narrower weight, where make_head_norm saw one
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("offset", ctypes.c_float)]


class Kv8Codes(ctypes.Structure):
    shape = None  # (pages, key heads, page size, head dim), where make_kv8_cache saw tensors
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_exp", ctypes.c_void_p),
                ("v_exp", ctypes.c_void_p)]


_lock = threading.Lock()
_lib = None
_raw_stream = None  # -> handle of the current stream


def load_library(path: str = LIB_PATH):
    """Load libgdn.so (raises if it was not built: there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing: build it with "
                              "`python -c 'import __graft_entry__ as g; g.build()'`")
        lib = ctypes.CDLL(path)
        P, I, S = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        D, B, PR = ctypes.POINTER(Dims), ctypes.POINTER(Batch), ctypes.POINTER(Params)
        AD, KB, RP = (ctypes.POINTER(AttnDims), ctypes.POINTER(KvBatch),
                      ctypes.POINTER(RopeParams))
        HN, KC = ctypes.POINTER(HeadNorm), ctypes.POINTER(Kv8Codes)
        L = ctypes.c_int64
        sig = {
            "gdn_page_layout": ([D, ctypes.POINTER(PageLayout)], I),
            "gdn_slot_layout": ([D, ctypes.POINTER(SlotLayout)], I),
            "gdn_conv": ([D, B, PR, P, P, P, I, P, P, P], I),
            "gdn_seq": ([D, B, PR, P, P, P, P, P, P, P], I),
            "gdn_spec_verify": ([D, B, PR, P, P, P, P, P, P, P], I),
            "gdn_spec_step": ([D, B, PR, P, P, P, P, P, P, P, P], I),
            "gdn_decode": ([D, B, PR, P, P, P, P, P, P, P, P], I),
            "gdn_prefill": ([D, B, PR, P, P, P, P, P, I, P, S, P, P], I),
            "gdn_spec_slots": ([D, B, PR, P, P, P, P, P, P, P, P, P], I),
            "gdn_page_to_slots": ([D, I, P, P, I, I, P, P, P, P], I),
            "gdn_slots_to_page": ([D, I, P, P, P, I, I, P, P, P, P], I),
            "gdn_chunk_prefill_workspace_bytes": ([D, B], S),
            "gdn_chunk_prefill": ([D, B, PR, P, P, P, P, P, P, S, P, P], I),
            "gdn_chunk_prefill_noalloc": ([D, B, PR, P, P, P, P, P, P, P], I),
            "gdn_check_bounded_wait": ([ctypes.c_int64, P, P], I),
            "gdn_rope": ([AD, RP, I, P, L, P, L, P, L, P, L, I, P], I),
            "gdn_kv_append": ([AD, KB, RP, P, L, P, L, P, L, P, L, P, P, P, P], I),
            "gdn_attn_plan_bytes": ([AD, KB], S),
            "gdn_attn_workspace_bytes": ([AD, KB], S),
            "gdn_attn_plan": ([AD, KB, P, S, P, P], I),
            "gdn_attn": ([AD, KB, P, P, L, P, P, P, P, P, S, P, P], I),
            "gdn_norm_rope": ([AD, HN, RP, I, P, L, P, L, P, L, P, L, P], I),
            "gdn_kv8_append": ([AD, KB, HN, RP, P, L, P, L, P, L, P, L, KC, P, P], I),
            "gdn_kv8_read": ([AD, KB, KC, P, L, P, L, P, P], I),
            "gdn_kv8_attn_plan_bytes": ([AD, KB], S),
            "gdn_kv8_attn_workspace_bytes": ([AD, KB], S),
            "gdn_kv8_attn_plan": ([AD, KB, P, S, P, P], I),
            "gdn_kv8_attn": ([AD, KB, P, P, L, KC, P, P, P, S, P, P], I),
            "gdn_strerror": ([I], ctypes.c_char_p),
            "gdn_abi_version": ([], I),
        }
        for name, (args, res) in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
        return lib


# ------------------------------------------------------------- marshalling

def _ptr(t):
    """Device/host address of a torch tensor (or an int address, or None)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        # the handle alone: building a Stream object costs as much as a launch
        global _raw_stream
        if _raw_stream is None:
            import torch
            raw, device = (getattr(torch._C, n, None) for n in
                           ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
            if raw is not None and device is not None:
                torch.cuda.init()
                _raw_stream = lambda: raw(device())  # noqa: E731
            else:
                _raw_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
        return _raw_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(code, where):
    if code != 0:
        raise GdnError(code, where)


def make_dims(Hk, Hv, Dk, Dv, W=4, Kc=0, io=GDN_BF16, state=GDN_F32, out=GDN_BF16) -> Dims:
    return Dims(Hk, Hv, Dk, Dv, W, Kc, io, state, out)


def make_params(A_log, dt_bias, conv_bias=None, scale=0.0, norm_eps=1e-6, gate_mode=0) -> Params:
    return Params(_ptr(A_log), _ptr(dt_bias), _ptr(conv_bias), float(scale), float(norm_eps),
                  int(gate_mode))


def make_batch(num_requests, num_rows, max_rows, num_pages, row_start, row_len, page, flags,
               n_accepted=None, order=None) -> Batch:
    """Row map from device int32 tensors (flags may be int32 or uint32 bits)."""
    return Batch(int(num_requests), int(num_rows), int(max_rows), int(num_pages), _ptr(row_start),
                 _ptr(row_len), _ptr(page), _ptr(flags), _ptr(n_accepted), _ptr(order))


def gdn_page_layout(dims: Dims) -> PageLayout:
    out = PageLayout()
    _check(load_library().gdn_page_layout(ctypes.byref(dims), ctypes.byref(out)), "gdn_page_layout")
    return out


def gdn_slot_layout(dims: Dims) -> SlotLayout:
    out = SlotLayout()
    _check(load_library().gdn_slot_layout(ctypes.byref(dims), ctypes.byref(out)), "gdn_slot_layout")
    return out


def gdn_conv(dims, batch, params, x, conv_w, y, y_dtype, pages, status, stream=None):
    _check(load_library().gdn_conv(ctypes.byref(dims), ctypes.byref(batch), ctypes.byref(params),
                                   _ptr(x), _ptr(conv_w), _ptr(y), int(y_dtype), _ptr(pages),
                                   _ptr(status), _stream(stream)), "gdn_conv")


def gdn_seq(dims, batch, params, qkv, a, b, o, pages, status, stream=None):
    _check(load_library().gdn_seq(ctypes.byref(dims), ctypes.byref(batch), ctypes.byref(params),
                                  _ptr(qkv), _ptr(a), _ptr(b), _ptr(o), _ptr(pages), _ptr(status),
                                  _stream(stream)), "gdn_seq")


def gdn_decode(dims, batch, params, x, conv_w, a, b, o, pages, status, stream=None):
    _check(load_library().gdn_decode(ctypes.byref(dims), ctypes.byref(batch), ctypes.byref(params),
                                     _ptr(x), _ptr(conv_w), _ptr(a), _ptr(b), _ptr(o), _ptr(pages),
                                     _ptr(status), _stream(stream)), "gdn_decode")


def gdn_prefill(dims, batch, params, qkv, a, b, o, pages, status, chunk_min_rows=0, stream=None,
                workspace=None, workspace_bytes=0):
    _check(load_library().gdn_prefill(ctypes.byref(dims), ctypes.byref(batch), ctypes.byref(params),
                                      _ptr(qkv), _ptr(a), _ptr(b), _ptr(o), _ptr(pages),
                                      int(chunk_min_rows), _ptr(workspace), int(workspace_bytes),
                                      _ptr(status), _stream(stream)),
           "gdn_prefill")


def gdn_spec_verify(dims, batch, params, qkv, a, b, o, pages, status, stream=None):
    _check(load_library().gdn_spec_verify(ctypes.byref(dims), ctypes.byref(batch),
                                          ctypes.byref(params), _ptr(qkv), _ptr(a), _ptr(b),
                                          _ptr(o), _ptr(pages), _ptr(status), _stream(stream)),
           "gdn_spec_verify")


def gdn_spec_step(dims, batch, params, x, conv_w, a, b, o, pages, status, stream=None):
    _check(load_library().gdn_spec_step(ctypes.byref(dims), ctypes.byref(batch),
                                        ctypes.byref(params), _ptr(x), _ptr(conv_w), _ptr(a),
                                        _ptr(b), _ptr(o), _ptr(pages), _ptr(status),
                                        _stream(stream)), "gdn_spec_step")


def gdn_spec_slots(dims, batch, params, x, conv_w, y, a, b, o, slots, status, stream=None):
    _check(load_library().gdn_spec_slots(ctypes.byref(dims), ctypes.byref(batch),
                                         ctypes.byref(params), _ptr(x), _ptr(conv_w), _ptr(y),
                                         _ptr(a), _ptr(b), _ptr(o), _ptr(slots), _ptr(status),
                                         _stream(stream)), "gdn_spec_slots")


def gdn_page_to_slots(dims, n, page, pool, num_pages, num_pools, pages, slots, status,
                      stream=None):
    _check(load_library().gdn_page_to_slots(ctypes.byref(dims), int(n), _ptr(page), _ptr(pool),
                                            int(num_pages), int(num_pools), _ptr(pages),
                                            _ptr(slots), _ptr(status), _stream(stream)),
           "gdn_page_to_slots")


def gdn_slots_to_page(dims, n, pool, slot, page, num_pools, num_pages, slots, pages, status,
                      stream=None):
    _check(load_library().gdn_slots_to_page(ctypes.byref(dims), int(n), _ptr(pool), _ptr(slot),
                                            _ptr(page), int(num_pools), int(num_pages),
                                            _ptr(slots), _ptr(pages), _ptr(status),
                                            _stream(stream)), "gdn_slots_to_page")


def gdn_chunk_prefill_workspace_bytes(dims, batch) -> int:
    return int(load_library().gdn_chunk_prefill_workspace_bytes(ctypes.byref(dims),
                                                                 ctypes.byref(batch)))


def gdn_chunk_prefill(dims, batch, params, qkv, a, b, o, pages, workspace, workspace_bytes,
                      status, stream=None):
    _check(load_library().gdn_chunk_prefill(ctypes.byref(dims), ctypes.byref(batch),
                                            ctypes.byref(params), _ptr(qkv), _ptr(a), _ptr(b),
                                            _ptr(o), _ptr(pages), _ptr(workspace),
                                            int(workspace_bytes), _ptr(status), _stream(stream)),
           "gdn_chunk_prefill")


def gdn_chunk_prefill_noalloc(dims, batch, params, qkv, a, b, o, pages, status, stream=None):
    _check(load_library().gdn_chunk_prefill_noalloc(ctypes.byref(dims), ctypes.byref(batch),
                                                    ctypes.byref(params), _ptr(qkv), _ptr(a),
                                                    _ptr(b), _ptr(o), _ptr(pages), _ptr(status),
                                                    _stream(stream)),
           "gdn_chunk_prefill_noalloc")


def make_attn_dims(Hq, Hkv, D, page_size, io=GDN_BF16, scale=0.0) -> AttnDims:
    return AttnDims(Hq, Hkv, D, page_size, io, float(scale))


def _int32(t, least, what):
    """Address of a device int32 tensor of at least `least` contiguous elements (or None, or an
    int address)."""
    if t is None or isinstance(t, int):
        return t
    import torch
    if t.dtype is not torch.int32 or t.numel() < least or not t.is_contiguous():
        _refuse(f"{what}: {t.dtype} {tuple(t.shape)} strides {t.stride()} where {least} int32 "
                "values side by side are read")
    return t.data_ptr()


def make_rope(rotary_dim, inv_freq, positions, axis=None, interleaved=False) -> RopeParams:
    """positions: device int32 [rows] or [axes][rows]; axis: device int32 [rotary_dim / 2];
    inv_freq: device float32 [rotary_dim / 2]. The structure keeps its tensors."""
    rotary_dim = int(rotary_dim)
    axes = 1 if positions is None or positions.dim() == 1 else positions.shape[0]
    if inv_freq is not None and not isinstance(inv_freq, int):
        import torch
        if (inv_freq.dtype is not torch.float32 or inv_freq.numel() < rotary_dim // 2
                or not inv_freq.is_contiguous()):
            _refuse(f"inv_freq: {inv_freq.dtype} {tuple(inv_freq.shape)} where "
                    f"{rotary_dim // 2} float32 values side by side are read")
    rope = RopeParams(rotary_dim, int(axes), int(interleaved), _ptr(inv_freq),
                      _int32(axis, rotary_dim // 2, "axis"), _int32(positions, 0, "positions"))
    rope.tensors = (inv_freq, axis, positions)
    rope.columns = None if positions is None else int(positions.shape[-1])
    return rope


def make_kv_batch(num_requests, num_rows, max_rows, num_pages, row_start, row_len, kv_len,
                  page_table, group_start=None, group_len=None, group_pages=None) -> KvBatch:
    """Row map over a paged cache from device int32 tensors; page_table [requests][pages]. The
    structure keeps its tensors."""
    R, width = int(num_requests), 0 if page_table is None else int(page_table.shape[1])
    groups = 0 if group_start is None else int(group_start.numel())
    batch = KvBatch(R, int(num_rows), int(max_rows), int(num_pages), width, groups,
                    _int32(row_start, R, "row_start"), _int32(row_len, R, "row_len"),
                    _int32(kv_len, R, "kv_len"), _int32(page_table, R * width, "page_table"),
                    _int32(group_start, groups, "group_start"),
                    _int32(group_len, groups, "group_len"),
                    _int32(group_pages, groups, "group_pages"))
    batch.tensors = (row_start, row_len, kv_len, page_table, group_start, group_len, group_pages)
    return batch


class _Types(dict):
    """dtype code -> torch dtype; None for other codes, which the calls themselves refuse."""

    def __missing__(self, code):
        import torch
        self.update({GDN_F32: torch.float32, GDN_BF16: torch.bfloat16, GDN_F16: torch.float16})
        return self.get(code)


_types = _Types()
# Several fields of a structure in one go (a field by itself costs half as much as all)
_attn_dims = struct.Struct("=5i").unpack_from   # (Hq, Hkv, D, page size, io dtype)
_kv_counts = struct.Struct("=4i").unpack_from   # (requests, rows, max rows, pages)


def _refuse(what):
    raise GdnError(CODES["GDN_ERR_INVALID_ARG"], what)


def _rows(t, heads, dim, dtype):
    """(rows, address, elements between rows) of a [rows][heads][dim] tensor whose heads are
    contiguous within a row, e.g. a slice of a projection's output. It may have more heads than
    the call takes."""
    n, h, d = t.shape
    if h < heads or d != dim or (t.dtype is not dtype and dtype is not None):
        _refuse(f"row tensor: {t.dtype} {tuple(t.shape)} for {heads} heads x {dim} of {dtype}")
    if t.is_contiguous():
        return n, t.data_ptr(), h * d
    between, head, one = t.stride()
    if one != 1 or (h > 1 and head != d):
        _refuse("row tensor: heads not contiguous")
    return n, t.data_ptr(), (between if n > 1 else h * d)


def _too_few(what, n, rows):
    _refuse(f"{what}: {n} rows where {rows} are used")


def _dense(t, count, dtype, what):
    """Address of a tensor of at least `count` contiguous elements (or None, or an int address)."""
    if t is None or isinstance(t, int):
        return t
    if (t.dtype is not dtype and dtype is not None) or t.numel() < count or not t.is_contiguous():
        _refuse(f"{what}: {t.dtype} {tuple(t.shape)} strides {t.stride()} where {count} elements of "
                f"{dtype} side by side are used")
    return t.data_ptr()


def _positions(rope, rows):
    """rope.columns differs from the call's rows: more are all right on a single axis."""
    n = rope.columns
    if n is not None and (n < rows or rope.num_axes > 1) and rope.rotary_dim:
        _refuse(f"positions: {n} on each axis for {rows} rows")


def gdn_rope(dims, rope, q, q_out, k=None, k_out=None, inverse=False, stream=None):
    hq, hk, dim, _, io = _attn_dims(dims)
    dtype = _types[io]
    q_at = q_row = qo_at = qo_row = k_at = k_row = ko_at = ko_row = 0
    if q is None and k is None:
        _refuse("gdn_rope: neither q nor k")
    if q is not None:
        rows, q_at, q_row = _rows(q, hq, dim, dtype)
    if k is not None:
        n, k_at, k_row = _rows(k, hk, dim, dtype)
        if q is not None and n != rows:
            _refuse(f"gdn_rope: q has {rows} rows, k {n}")
        rows = n
    if q_out is not None:
        n, qo_at, qo_row = _rows(q_out, hq, dim, dtype)
        if n < rows:
            _too_few("q_out", n, rows)
    if k_out is not None:
        n, ko_at, ko_row = _rows(k_out, hk, dim, dtype)
        if n < rows:
            _too_few("k_out", n, rows)
    if rope.columns != rows:
        _positions(rope, rows)
    # (a structure passed where a pointer is declared goes by reference)
    code = (_lib or load_library()).gdn_rope(dims, rope, rows, q_at, q_row, qo_at, qo_row, k_at,
                                             k_row, ko_at, ko_row, int(inverse), _stream(stream))
    if code:
        raise GdnError(code, "gdn_rope")


def gdn_kv_append(dims, batch, rope, q, k, v, q_out, k_cache, v_cache, status, stream=None):
    hq, hk, dim, ps, io = _attn_dims(dims)
    _, rows, _, pages = _kv_counts(batch)
    dtype, n_cache = _types[io], pages * hk * ps * dim
    q_at = q_row = qo_at = qo_row = k_at = k_row = v_at = v_row = 0
    if k is not None:
        n, k_at, k_row = _rows(k, hk, dim, dtype)
        if n < rows:
            _too_few("k", n, rows)
    if v is not None:
        n, v_at, v_row = _rows(v, hk, dim, dtype)
        if n < rows:
            _too_few("v", n, rows)
    if q is not None:
        n, q_at, q_row = _rows(q, hq, dim, dtype)
        if n < rows:
            _too_few("q", n, rows)
    if q_out is not None:
        n, qo_at, qo_row = _rows(q_out, hq, dim, dtype)
        if n < rows:
            _too_few("q_out", n, rows)
    if rope is not None and rope.columns != rows:
        _positions(rope, rows)
    code = (_lib or load_library()).gdn_kv_append(
        dims, batch, rope, q_at, q_row, k_at, k_row, v_at, v_row, qo_at, qo_row,
        _dense(k_cache, n_cache, dtype, "k_cache"), _dense(v_cache, n_cache, dtype, "v_cache"),
        _ptr(status), _stream(stream))
    if code:
        raise GdnError(code, "gdn_kv_append")


def gdn_attn_plan_bytes(dims, batch) -> int:
    return int(load_library().gdn_attn_plan_bytes(ctypes.byref(dims), ctypes.byref(batch)))


def gdn_attn_workspace_bytes(dims, batch) -> int:
    return int(load_library().gdn_attn_workspace_bytes(ctypes.byref(dims), ctypes.byref(batch)))


def gdn_attn_plan(dims, batch, plan, plan_bytes, status, stream=None):
    _check(load_library().gdn_attn_plan(ctypes.byref(dims), ctypes.byref(batch), _ptr(plan),
                                        int(plan_bytes), _ptr(status), _stream(stream)),
           "gdn_attn_plan")


def gdn_attn(dims, batch, plan, q, k_cache, v_cache, o, lse, workspace, workspace_bytes, status,
             stream=None):
    hq, hk, dim, ps, io = _attn_dims(dims)
    _, rows, _, pages = _kv_counts(batch)
    dtype, n_cache, q_at, q_row = _types[io], pages * hk * ps * dim, 0, 0
    if q is not None:
        n, q_at, q_row = _rows(q, hq, dim, dtype)
        if n < rows:
            _too_few("q", n, rows)
    code = (_lib or load_library()).gdn_attn(
        dims, batch, _ptr(plan), q_at, q_row, _dense(k_cache, n_cache, dtype, "k_cache"),
        _dense(v_cache, n_cache, dtype, "v_cache"), _dense(o, rows * hq * dim, dtype, "o"),
        _dense(lse, rows * hq, _types[GDN_F32], "lse"), _ptr(workspace), int(workspace_bytes),
        _ptr(status), _stream(stream))
    if code:
        raise GdnError(code, "gdn_attn")


def make_head_norm(q_weight=None, k_weight=None, eps=1e-6, offset=0.0) -> HeadNorm:
    """RMS norm of each head: x / sqrt(mean x^2 + eps) * (offset + weight); weights: device
    float32 [D] or None. The structure keeps its tensors."""
    width = None
    for w, what in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is None or isinstance(w, int):
            continue
        import torch
        if w.dtype is not torch.float32 or not w.is_contiguous():
            _refuse(f"{what}: {w.dtype} strides {w.stride()} where float32 values side by side "
                    "are read")
        width = w.numel() if width is None else min(width, w.numel())
    norm = HeadNorm(_ptr(q_weight), _ptr(k_weight), float(eps), float(offset))
    norm.tensors, norm.width = (q_weight, k_weight), width
    return norm


def make_kv8_cache(k, v, k_exp, v_exp) -> Kv8Codes:
    """A cache of 8-bit codes: k, v float8_e4m3fn or uint8 [pages][Hkv][page size][D], k_exp,
    v_exp int8 [pages][Hkv][page size / 16]; device, contiguous (k or v may be None where only
    the other is read). The structure keeps its tensors."""
    shape = None
    for codes, exps, what in ((k, k_exp, "k"), (v, v_exp, "v")):
        if codes is None or isinstance(codes, int):
            continue
        import torch
        if (codes.dtype not in (torch.float8_e4m3fn, torch.uint8) or codes.dim() != 4
                or not codes.is_contiguous()):
            _refuse(f"{what}: {codes.dtype} {tuple(codes.shape)} strides {codes.stride()} where "
                    "dense codes [pages][heads][page size][D] are used")
        pages, heads, ps, _ = codes.shape
        if (exps is None or isinstance(exps, int) or exps.dtype is not torch.int8
                or tuple(exps.shape) != (pages, heads, ps // 16) or not exps.is_contiguous()):
            _refuse(f"{what}_exp: int8 [{pages}][{heads}][{ps // 16}], dense, goes with {what}")
        if shape is not None and tuple(codes.shape) != shape:
            _refuse(f"k {shape} and v {tuple(codes.shape)} differ")
        shape = tuple(codes.shape)
    cache = Kv8Codes(_ptr(k), _ptr(v), _ptr(k_exp), _ptr(v_exp))
    cache.tensors, cache.shape = (k, v, k_exp, v_exp), shape
    return cache


def _kv8_fits(cache, hk, ps, dim, pages):
    if cache is None:
        _refuse("no cache")
    shape = cache.shape
    if shape is not None and (shape[0] < pages or shape[1:] != (hk, ps, dim)):
        _refuse(f"cache {shape} where [{pages}][{hk}][{ps}][{dim}] is used")


def _norm_fits(norm, dim):
    if norm is not None and norm.width is not None and norm.width < dim:
        _refuse(f"norm weights of {norm.width} elements for heads of {dim}")


def gdn_norm_rope(dims, norm, rope, q, q_out, k=None, k_out=None, stream=None):
    hq, hk, dim, _, io = _attn_dims(dims)
    dtype = _types[io]
    q_at = q_row = qo_at = qo_row = k_at = k_row = ko_at = ko_row = 0
    if q is None and k is None:
        _refuse("gdn_norm_rope: neither q nor k")
    _norm_fits(norm, dim)
    if q is not None:
        rows, q_at, q_row = _rows(q, hq, dim, dtype)
    if k is not None:
        n, k_at, k_row = _rows(k, hk, dim, dtype)
        if q is not None and n != rows:
            _refuse(f"gdn_norm_rope: q has {rows} rows, k {n}")
        rows = n
    if q_out is not None:
        n, qo_at, qo_row = _rows(q_out, hq, dim, dtype)
        if n < rows:
            _too_few("q_out", n, rows)
    if k_out is not None:
        n, ko_at, ko_row = _rows(k_out, hk, dim, dtype)
        if n < rows:
            _too_few("k_out", n, rows)
    if rope is not None and rope.columns != rows:
        _positions(rope, rows)
    code = (_lib or load_library()).gdn_norm_rope(dims, norm, rope, rows, q_at, q_row, qo_at,
                                                  qo_row, k_at, k_row, ko_at, ko_row,
                                                  _stream(stream))
    if code:
        raise GdnError(code, "gdn_norm_rope")


def gdn_kv8_append(dims, batch, norm, rope, q, k, v, q_out, cache, status, stream=None):
    hq, hk, dim, ps, io = _attn_dims(dims)
    _, rows, _, pages = _kv_counts(batch)
    dtype = _types[io]
    q_at = q_row = qo_at = qo_row = k_at = k_row = v_at = v_row = 0
    _kv8_fits(cache, hk, ps, dim, pages)
    _norm_fits(norm, dim)
    if k is not None:
        n, k_at, k_row = _rows(k, hk, dim, dtype)
        if n < rows:
            _too_few("k", n, rows)
    if v is not None:
        n, v_at, v_row = _rows(v, hk, dim, dtype)
        if n < rows:
            _too_few("v", n, rows)
    if q is not None:
        n, q_at, q_row = _rows(q, hq, dim, dtype)
        if n < rows:
            _too_few("q", n, rows)
    if q_out is not None:
        n, qo_at, qo_row = _rows(q_out, hq, dim, dtype)
        if n < rows:
            _too_few("q_out", n, rows)
    if rope is not None and rope.columns != rows:
        _positions(rope, rows)
    code = (_lib or load_library()).gdn_kv8_append(
        dims, batch, norm, rope, q_at, q_row, k_at, k_row, v_at, v_row, qo_at, qo_row, cache,
        _ptr(status), _stream(stream))
    if code:
        raise GdnError(code, "gdn_kv8_append")


def gdn_kv8_read(dims, batch, cache, k_out, v_out, status, stream=None):
    hq, hk, dim, ps, io = _attn_dims(dims)
    _, rows, _, pages = _kv_counts(batch)
    dtype = _types[io]
    k_at = k_row = v_at = v_row = 0
    _kv8_fits(cache, hk, ps, dim, pages)
    if k_out is not None:
        n, k_at, k_row = _rows(k_out, hk, dim, dtype)
        if n < rows:
            _too_few("k_out", n, rows)
    if v_out is not None:
        n, v_at, v_row = _rows(v_out, hk, dim, dtype)
        if n < rows:
            _too_few("v_out", n, rows)
    code = (_lib or load_library()).gdn_kv8_read(dims, batch, cache, k_at, k_row, v_at, v_row,
                                                 _ptr(status), _stream(stream))
    if code:
        raise GdnError(code, "gdn_kv8_read")


def gdn_kv8_attn_plan_bytes(dims, batch) -> int:
    return int(load_library().gdn_kv8_attn_plan_bytes(ctypes.byref(dims), ctypes.byref(batch)))


def gdn_kv8_attn_workspace_bytes(dims, batch) -> int:
    return int(load_library().gdn_kv8_attn_workspace_bytes(ctypes.byref(dims),
                                                           ctypes.byref(batch)))


def gdn_kv8_attn_plan(dims, batch, plan, plan_bytes, status, stream=None):
    _check(load_library().gdn_kv8_attn_plan(ctypes.byref(dims), ctypes.byref(batch), _ptr(plan),
                                            int(plan_bytes), _ptr(status), _stream(stream)),
           "gdn_kv8_attn_plan")


def gdn_kv8_attn(dims, batch, plan, q, cache, o, lse, workspace, workspace_bytes, status,
                 stream=None):
    hq, hk, dim, ps, io = _attn_dims(dims)
    _, rows, _, pages = _kv_counts(batch)
    dtype, q_at, q_row = _types[io], 0, 0
    _kv8_fits(cache, hk, ps, dim, pages)
    if q is not None:
        n, q_at, q_row = _rows(q, hq, dim, dtype)
        if n < rows:
            _too_few("q", n, rows)
    code = (_lib or load_library()).gdn_kv8_attn(
        dims, batch, _ptr(plan), q_at, q_row, cache, _dense(o, rows * hq * dim, dtype, "o"),
        _dense(lse, rows * hq, _types[GDN_F32], "lse"), _ptr(workspace), int(workspace_bytes),
        _ptr(status), _stream(stream))
    if code:
        raise GdnError(code, "gdn_kv8_attn")


def gdn_check_bounded_wait(limit_ns, status, stream=None):
    _check(load_library().gdn_check_bounded_wait(int(limit_ns), _ptr(status), _stream(stream)),
           "gdn_check_bounded_wait")


def gdn_strerror(code: int) -> str:
    return load_library().gdn_strerror(int(code)).decode()


def gdn_abi_version() -> int:
    return int(load_library().gdn_abi_version())


def raise_on_status(status, where="device"):
    """Read the device status word (synchronises its stream) and raise if set."""
    code = int(status.item())
    if code != 0:
        raise GdnError(code, where)
