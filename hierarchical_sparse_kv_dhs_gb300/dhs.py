"""ctypes binding of libdhs (include/dhs.h): same names, argument marshalling
only.  Every step of the resolve + gather path runs in the library's CUDA
kernels; nothing here computes a location, a victim or a byte.

PyTorch supplies device memory and streams; pinned host rows come from
``HostRows`` (page-aligned anonymous memory registered as mapped pinned
memory with the CUDA runtime).

Importing this module fails loudly when libdhs.so has not been built.
"""
from __future__ import annotations

import ctypes
import functools
import mmap
import os
import struct
import sys

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdhs.so")

DHS_OK = 0
DHS_EINVAL = -1
DHS_ENOMEM = -2
DHS_EWOULDWAIT = -3
DHS_EBUDGET = -4
DHS_ERANGE = -5
DHS_ETIMEDOUT = -6
DHS_ECUDA = -7
DHS_ESTATE = -8
RC_NAMES = {0: 0, -1: "einval", -2: "enomem", -3: "wouldwait", -4: "ebudget",
            -5: "erange", -6: "etimedout", -7: "ecuda", -8: "estate"}

DHS_TIER_TAIL, DHS_TIER_OPT, DHS_TIER_HOT = 0, 1, 2
DHS_NO_LOC = 0xFFFFFFFF
DHS_END_LOC = 0xFFFFFFFE
DHS_NUM_COUNTERS = 8
DHS_STATUS_ERANGE, DHS_STATUS_EBUDGET, DHS_STATUS_ELOC, DHS_STATUS_ETIMEDOUT = 1, 2, 4, 8
DHS_ITEM_GATHER_ONLY = 1
DHS_ITEM_UNION = 2
DHS_OPT_COPY_CTAS = 1
DHS_OPT_GATHER_IMPL = 2
DHS_OPT_TRACE = 3
DHS_OPT_EARLY = 4
DHS_OPT_FRESH_LIST = 5
DHS_OPT_GATHER_TPC = 6
DHS_OPT_STAGE_MISSES = 7
DHS_OPT_MARK_POLLS = 8
DHS_OPT_COPY_PDL = 9
DHS_OPT_RESOLVE_PAIRED = 10
DHS_OPT_COPY_STEAL = 11
DHS_OPT_RESOLVE_CTAS = 12
DHS_OPT_ATTEND_POLLS = 13
DHS_BF16, DHS_F16 = 0, 1
DHS_ATTEND_HISTORY = 1
DHS_ATTEND_MAX_KEY, DHS_ATTEND_MAX_VALUE = 576, 512
DHS_ROPE_PLAIN, DHS_ROPE_LINEAR, DHS_ROPE_BASE, DHS_ROPE_PARTS = range(4)
DHS_ROPE_HALF, DHS_ROPE_INTERLEAVED = 0, 1
DHS_ROPE_INVERSE = 1
DHS_PACKED_MAX_WIDE = 64
DHS_UNPACK_HISTORY = 1
DHS_BUF_HOT, DHS_BUF_TAIL, DHS_BUF_OPT, DHS_BUF_META = range(4)

_i32, _i64, _u32, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_void_p


class dhs_pool_config(ctypes.Structure):
    _fields_ = [("max_requests", _i32), ("sources", _i32), ("row_bytes", _i32),
                ("page_rows", _i32), ("tail_rows", _i32), ("hot_rows", _i32),
                ("max_queries", _i32), ("max_topk", _i32),
                ("max_rows_per_request", _i64), ("optional_pages", _i64),
                ("admission_reserve_pages", _i64),
                ("hot_dev", _vp), ("tail_dev", _vp), ("opt_dev", _vp),
                ("meta_dev", _vp), ("stream", _vp)]


class dhs_append_item(ctypes.Structure):
    _fields_ = [("req", _i32), ("src", _i32), ("count", _i32), ("reserved", _i32),
                ("rows_dev", _vp)]


class dhs_item(ctypes.Structure):
    _fields_ = [("req", _i32), ("src", _i32), ("queries", _i32), ("topk", _i32),
                ("flags", _u32), ("reserved", _i32), ("sel_dev", _vp),
                ("loc_dev", _vp), ("staging_dev", _vp), ("counters_dev", _vp),
                ("index_dev", _vp)]


class dhs_copy(ctypes.Structure):
    _fields_ = [("dst", _vp), ("src", _vp), ("bytes", ctypes.c_size_t)]


class dhs_attend_item(ctypes.Structure):
    _fields_ = [("req", _i32), ("src", _i32), ("queries", _i32), ("topk", _i32),
                ("flags", _u32), ("reserved", _i32), ("q_dev", _vp), ("loc_dev", _vp),
                ("index_dev", _vp), ("range_dev", _vp), ("out_dev", _vp), ("lse_dev", _vp)]


class dhs_attend_step(ctypes.Structure):
    _fields_ = [("n_items", _i32), ("dtype", _i32), ("heads", _i32), ("kv_heads", _i32),
                ("key_elems", _i32), ("value_elems", _i32), ("key_offset", _i32),
                ("value_offset", _i32), ("key_stride", _i32), ("value_stride", _i32),
                ("scale", ctypes.c_float), ("reserved", _i32),
                ("q_query_stride", _i64), ("q_head_stride", _i64),
                ("out_query_stride", _i64), ("out_head_stride", _i64),
                ("items", ctypes.POINTER(dhs_attend_item)), ("work_dev", _vp),
                ("work_bytes", ctypes.c_size_t)]


_f64, _f32 = ctypes.c_double, ctypes.c_float


class dhs_rope_config(ctypes.Structure):
    _fields_ = [("rotary_elems", _i32), ("scaling", _i32), ("base", _f64), ("factor", _f64),
                ("original", _f64), ("fast", _f64), ("slow", _f64)]


class dhs_rotate_step(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("tokens", _i32), ("heads", _i32), ("head_elems", _i32),
                ("rotary_offset", _i32), ("rotary_elems", _i32), ("pairs", _i32), ("flags", _u32),
                ("amplitude", _f32), ("reserved", _i32), ("x_token_stride", _i64),
                ("x_head_stride", _i64), ("y_token_stride", _i64), ("y_head_stride", _i64),
                ("x_dev", _vp), ("y_dev", _vp), ("position_dev", _vp), ("turns_dev", _vp)]


class dhs_packed_rows(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("kv_heads", _i32), ("key_elems", _i32), ("wide_elems", _i32),
                ("value_elems", _i32), ("shared", _i32)]


class dhs_pack_item(ctypes.Structure):
    __slots__ = ("given",)
    _fields_ = [("req", _i32), ("src", _i32), ("count", _i32), ("reserved", _i32),
                ("key_dev", _vp), ("wide_dev", _vp), ("value_dev", _vp), ("position_dev", _vp),
                ("rows_dev", _vp)]


class dhs_pack_step(ctypes.Structure):
    _fields_ = [("rows", dhs_packed_rows), ("n_items", _i32), ("rotary_offset", _i32),
                ("rotary_elems", _i32), ("pairs", _i32), ("amplitude", _f32), ("reserved", _i32),
                ("key_token_stride", _i64), ("key_head_stride", _i64),
                ("wide_token_stride", _i64), ("wide_head_stride", _i64),
                ("value_token_stride", _i64), ("value_head_stride", _i64),
                ("turns_dev", _vp), ("items", ctypes.POINTER(dhs_pack_item))]


class dhs_unpack_item(ctypes.Structure):
    __slots__ = ("given",)
    _fields_ = [("req", _i32), ("src", _i32), ("count", _i32), ("flags", _u32), ("first", _i64),
                ("loc_dev", _vp), ("rows_dev", _vp), ("key_dev", _vp), ("value_dev", _vp)]


class dhs_unpack_step(ctypes.Structure):
    _fields_ = [("rows", dhs_packed_rows), ("n_items", _i32), ("reserved", _i32),
                ("key_row_stride", _i64), ("key_head_stride", _i64),
                ("value_row_stride", _i64), ("value_head_stride", _i64),
                ("items", ctypes.POINTER(dhs_unpack_item))]


class dhs_attend_packed_step(ctypes.Structure):
    _fields_ = [("rows", dhs_packed_rows), ("n_items", _i32), ("heads", _i32), ("scale", _f32),
                ("reserved", _i32), ("q_query_stride", _i64), ("q_head_stride", _i64),
                ("out_query_stride", _i64), ("out_head_stride", _i64),
                ("items", ctypes.POINTER(dhs_attend_item)), ("work_dev", _vp),
                ("work_bytes", ctypes.c_size_t)]


class dhs_step(ctypes.Structure):
    _fields_ = [("step", _u32), ("n_items", _i32), ("items", ctypes.POINTER(dhs_item))]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run hierarchical_sparse_kv_dhs_gb300.build.build() "
            "(nvcc, sm_103a) first -- there is no fallback path")
    L = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER
    sig = {
        "dhs_pool_bytes": (ctypes.c_int, [P(dhs_pool_config), P(ctypes.c_size_t)]),
        "dhs_pool_create": (ctypes.c_int, [P(dhs_pool_config), P(_vp)]),
        "dhs_pool_destroy": (None, [_vp]),
        "dhs_admit": (ctypes.c_int, [_vp, _i32, _i32, _vp, _i64, _vp, P(_i64)]),
        "dhs_reclaim": (ctypes.c_int, [_vp, _vp, _i32, _i64, P(_i64)]),
        "dhs_release": (ctypes.c_int, [_vp, _i32]),
        "dhs_prefetch": (ctypes.c_int, [_vp, _vp, _vp]),
        "dhs_gather_on": (ctypes.c_int, [_vp, _vp, _vp]),
        "dhs_decode_step_host": (ctypes.c_int, [_vp, _vp, _i32, _vp, _i32, _vp, _vp, _i32]),
        "dhs_decode_step_host_async": (ctypes.c_int, [_vp, _vp, _i32, _vp, _vp, _i32, _vp,
                                                      _vp, _i32, _vp]),
        "dhs_admit_device": (ctypes.c_int, [_vp, _i32, _i32, _vp, _vp, _i64, _vp, P(_i64)]),
        "dhs_admit_window": (ctypes.c_int, [_vp, _i32, _i32, _vp, _i64]),
        "dhs_backup": (ctypes.c_int, [_vp, _i64, P(_i64)]),
        "dhs_pending_backup": (_i64, [_vp]),
        "dhs_refill": (ctypes.c_int, [_vp, _i64, P(_i64)]),
        "dhs_pool_used": (_i64, [_vp]),
        "dhs_flush": (ctypes.c_int, [_vp]),
        "dhs_append": (ctypes.c_int, [_vp, P(dhs_append_item), _i32]),
        "dhs_resolve": (ctypes.c_int, [_vp, P(dhs_step)]),
        "dhs_gather": (ctypes.c_int, [_vp, P(dhs_step)]),
        "dhs_resolve_gather": (ctypes.c_int, [_vp, P(dhs_step)]),
        "dhs_resolve_noalloc": (ctypes.c_int, [_vp, P(dhs_step)]),
        "dhs_decode_step": (ctypes.c_int, [_vp, P(dhs_append_item), _i32, P(dhs_step)]),
        "dhs_attend_bytes": (ctypes.c_int, [_vp, P(dhs_attend_step), P(ctypes.c_size_t)]),
        "dhs_attend": (ctypes.c_int, [_vp, P(dhs_attend_step)]),
        "dhs_attend_on": (ctypes.c_int, [_vp, P(dhs_attend_step), _vp]),
        "dhs_rope_table": (ctypes.c_int, [_vp, _vp]),
        "dhs_rotate": (ctypes.c_int, [_vp, P(dhs_rotate_step)]),
        "dhs_rotate_on": (ctypes.c_int, [_vp, P(dhs_rotate_step), _vp]),
        "dhs_packed_bytes": (ctypes.c_int, [_vp, P(_i32)]),
        "dhs_pack": (ctypes.c_int, [_vp, P(dhs_pack_step)]),
        "dhs_append_packed": (ctypes.c_int, [_vp, P(dhs_pack_step)]),
        "dhs_unpack": (ctypes.c_int, [_vp, P(dhs_unpack_step)]),
        "dhs_unpack_on": (ctypes.c_int, [_vp, P(dhs_unpack_step), _vp]),
        "dhs_attend_packed_bytes": (ctypes.c_int, [_vp, P(dhs_attend_packed_step),
                                                   P(ctypes.c_size_t)]),
        "dhs_attend_packed": (ctypes.c_int, [_vp, P(dhs_attend_packed_step)]),
        "dhs_attend_packed_on": (ctypes.c_int, [_vp, P(dhs_attend_packed_step), _vp]),
        "dhs_fork": (ctypes.c_int, [_vp, _i32, _i32, P(_vp), P(_vp), P(_i64)]),
        "dhs_compact": (ctypes.c_int, [_vp, _i64, P(_i64)]),
        "dhs_pool_capacity": (_i64, [_vp]),
        "dhs_status": (ctypes.c_int, [_vp, P(_u32)]),
        "dhs_read_state": (ctypes.c_int, [_vp, _i32, _i32, _vp, _vp, _vp, _vp]),
        "dhs_set_option": (ctypes.c_int, [_vp, _i32, _i64]),
        "dhs_get_option": (ctypes.c_int, [_vp, _i32, ctypes.POINTER(_i64)]),
        "dhs_strerror": (ctypes.c_char_p, [ctypes.c_int]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    return L


lib = _load()


class DhsError(RuntimeError):
    def __init__(self, code, what=""):
        self.code = code
        super().__init__(f"{what}: {lib.dhs_strerror(code).decode()} ({code})")


def check(code, what=""):
    if code != DHS_OK:
        raise DhsError(code, what)
    return code


# ------------------------------------------------------------ C-named calls

def dhs_pool_bytes(cfg: dhs_pool_config) -> list[int]:
    out = (ctypes.c_size_t * 4)()
    check(lib.dhs_pool_bytes(ctypes.byref(cfg), out), "dhs_pool_bytes")
    return list(out)


def dhs_pool_create(cfg: dhs_pool_config) -> int:
    h = _vp()
    check(lib.dhs_pool_create(ctypes.byref(cfg), ctypes.byref(h)), "dhs_pool_create")
    return h.value


def dhs_pool_destroy(h: int) -> None:
    lib.dhs_pool_destroy(h)


def dhs_admit(h, req, src, host_ptr, n_rows, mask=None):
    d = _i64(0)
    m = None
    if mask is not None:
        mask = np.ascontiguousarray(mask, np.uint8)
        m = mask.ctypes.data
    rc = lib.dhs_admit(h, req, src, host_ptr, n_rows, m, ctypes.byref(d))
    return rc, d.value


def dhs_reclaim(h, order, deficit):
    o = np.ascontiguousarray(order, np.int32)
    f = _i64(0)
    rc = lib.dhs_reclaim(h, o.ctypes.data if len(o) else None, len(o), deficit,
                         ctypes.byref(f))
    return rc, f.value


def dhs_release(h, req):
    return lib.dhs_release(h, req)


def dhs_admit_device(h, req, src, dev_ptr, host_ptr, n_rows, mask=None):
    d = _i64(0)
    m = None
    if mask is not None:
        mask = np.ascontiguousarray(mask, np.uint8)
        m = mask.ctypes.data
    rc = lib.dhs_admit_device(h, req, src, dev_ptr, host_ptr, n_rows, m, ctypes.byref(d))
    return rc, d.value


def dhs_admit_window(h, req, src, dev_ptr, n_rows):
    return lib.dhs_admit_window(h, req, src, dev_ptr, n_rows)


def dhs_backup(h, max_pages):
    n = _i64(0)
    rc = lib.dhs_backup(h, max_pages, ctypes.byref(n))
    return rc, n.value


def dhs_refill(h, max_pages):
    n = _i64(0)
    rc = lib.dhs_refill(h, max_pages, ctypes.byref(n))
    return rc, n.value


def dhs_pool_used(h):
    return lib.dhs_pool_used(h)


def dhs_flush(h):
    return lib.dhs_flush(h)


def dhs_append(h, items):
    arr = (dhs_append_item * max(1, len(items)))(*items)
    return lib.dhs_append(h, arr, len(items))


def make_step(step: int, items) -> tuple:
    """A dhs_step plus the item array that must stay alive with it."""
    arr = (dhs_item * max(1, len(items)))(*items)
    return dhs_step(step, len(items), arr), arr


def _address(t):
    if t is None or type(t) is int:
        return t
    try:
        return t.data_ptr()
    except AttributeError:
        return t


def attend_item(*, queries, q, out, req=0, src=0, topk=0, flags=0, loc=None, index=None,
                range_=None, lse=None) -> dhs_attend_item:
    """A dhs_attend_item from torch tensors (or device addresses)."""
    ptr = _address
    it = dhs_attend_item()
    it.req, it.src, it.queries, it.topk, it.flags = req, src, queries, topk, flags
    it.q_dev, it.out_dev, it.loc_dev = ptr(q), ptr(out), ptr(loc)
    it.index_dev, it.range_dev, it.lse_dev = ptr(index), ptr(range_), ptr(lse)
    return it


def make_attend(items, *, heads, key_elems, value_elems, scale, kv_heads=1, key_offset=0,
                value_offset=0, key_stride=None, value_stride=None, q_strides=None,
                out_strides=None, dtype="bf16") -> tuple:
    """A dhs_attend_step (without a workspace) plus the item array that must
    stay alive with it.  Strides are in elements: between kv heads (default:
    back to back) and (between queries, between heads) of the queries and the
    outputs (default: contiguous [Q][heads][elems])."""
    arr = (dhs_attend_item * max(1, len(items)))(*items)
    st = dhs_attend_step()
    st.n_items, st.items = len(items), arr
    st.dtype = {"bf16": DHS_BF16, "f16": DHS_F16}[dtype]
    st.heads, st.kv_heads, st.scale = heads, kv_heads, scale
    st.key_elems, st.value_elems = key_elems, value_elems
    st.key_offset, st.value_offset = key_offset, value_offset
    st.key_stride = key_elems if key_stride is None else key_stride
    st.value_stride = value_elems if value_stride is None else value_stride
    st.q_query_stride, st.q_head_stride = q_strides or (heads * key_elems, key_elems)
    st.out_query_stride, st.out_head_stride = out_strides or (heads * value_elems, value_elems)
    return st, arr


def dhs_attend_bytes(h, st: dhs_attend_step) -> int:
    n = ctypes.c_size_t(0)
    check(lib.dhs_attend_bytes(h, ctypes.byref(st), ctypes.byref(n)), "dhs_attend_bytes")
    return n.value


def dhs_attend(h, st: dhs_attend_step):
    return lib.dhs_attend(h, ctypes.byref(st))


def dhs_attend_on(h, st: dhs_attend_step, stream):
    return lib.dhs_attend_on(h, ctypes.byref(st), stream)


_DTYPES = {"bf16": DHS_BF16, "f16": DHS_F16}
_PAIRS = {"half": DHS_ROPE_HALF, "interleaved": DHS_ROPE_INTERLEAVED}
_SCALINGS = {"plain": DHS_ROPE_PLAIN, "linear": DHS_ROPE_LINEAR, "base": DHS_ROPE_BASE,
             "parts": DHS_ROPE_PARTS}


def rope_table(rotary, *, base=10000.0, scaling="plain", factor=1.0, original=0.0, fast=32.0,
               slow=1.0):
    """dhs_rope_table's turns as an int64 array (the bits of the uint64s), which
    torch.from_numpy takes: move it to the GPU once and hand it to make_rotate
    and make_pack.  (scaling="parts" weights pairs by their turns; a ramp over the
    pairs' numbers is a table of the caller's: see dhs_rope_config.)"""
    cfg = dhs_rope_config(rotary, _SCALINGS[scaling], base, factor, original, fast, slow)
    out = np.empty(max(1, rotary // 2), np.int64)
    check(lib.dhs_rope_table(ctypes.byref(cfg), out.ctypes.data), "dhs_rope_table")
    return out


@functools.lru_cache(maxsize=None)
def _type_name(dtype):
    return str(dtype).rpartition(".")[2]


_WIDE = {"bfloat16": "bf16", "float16": "f16"}
_TORCH_TYPES = {}
_TURNS = ("int64", "uint64")


def _torch_type(code):
    """torch's type of a layout's (there are no tensors to check without torch)."""
    if not _TORCH_TYPES and "torch" in sys.modules:
        torch = sys.modules["torch"]
        _TORCH_TYPES.update({DHS_BF16: torch.bfloat16, DHS_F16: torch.float16})
    return _TORCH_TYPES.get(code)


class _Parts:
    """Checks of the tensors that a call reads or writes (None and addresses pass):
    where they lie, their types, and that they hold what the call takes of them."""

    def __init__(self, layout=None):
        self.device = None  # that of the tensors so far
        if layout is not None:
            self.layout, self.kv, self.row_bytes = layout, layout.kv_heads, None
            self.dtype = _torch_type(layout.dtype)

    def reach(self, t, what):
        """Whether t is a tensor; ValueError where the GPU cannot reach it, or not the others'."""
        if t is None or not hasattr(t, "data_ptr"):
            return False
        if t.get_device() != self.device:
            self.place(t, what)
        return True

    def place(self, t, what):
        device = t.get_device()
        if device < 0:
            if not t.is_pinned():
                raise ValueError(f"{what}: a tensor on the GPU is needed")
        elif self.device is None:
            self.device = device
        else:
            raise ValueError(f"{what}: tensors on one GPU are needed")

    def entries(self, t, what, types, n):
        """A list of n entries."""
        if self.reach(t, what) and (_type_name(t.dtype) not in types or t.numel() < n or
                                    not t.is_contiguous()):
            raise ValueError(f"{what}: {n} contiguous entries of {types[0]} are needed")

    def heads(self, t, what, count, elems, strides):
        """`count` rows' heads of `elems` elements of the layout's type; strides
        None: contiguous ones."""
        if not self.reach(t, what):
            return
        if t.dtype is not self.dtype:
            raise ValueError(f"{what}: {t.dtype} is not the layout's type")
        if strides is None:
            if t.numel() < count * self.kv * elems or not t.is_contiguous():
                raise ValueError(f"{what}: contiguous [{count}][{self.kv}][{elems}] or strides are needed")
        elif count > 0:
            ends = [(n - 1) * s for n, s in zip((count, self.kv), strides)]
            first, size = t.storage_offset(), t.untyped_storage().nbytes() // t.element_size()
            if first + sum(min(0, e) for e in ends) < 0 or \
                    first + sum(max(0, e) for e in ends) + elems > size:
                raise ValueError(f"{what}: [{count}][{self.kv}][{elems}] by these strides leaves the tensor")

    def packed(self, t, count):
        """`count` packed rows (of a layout that is refused: the call says so)."""
        if t is None or not self.reach(t, "rows"):
            return
        if self.row_bytes is None:
            n = _i32(0)
            lib.dhs_packed_bytes(ctypes.byref(self.layout), ctypes.byref(n))
            self.row_bytes = n.value
        if t.numel() * t.element_size() < count * self.row_bytes or not t.is_contiguous():
            raise ValueError(f"rows: {count} contiguous rows of {self.row_bytes} bytes are needed")


def make_rotate(x, positions, turns, *, out=None, offset=0, rotary=None, pairs="half",
                inverse=False, amplitude=1.0) -> dhs_rotate_step:
    """A dhs_rotate_step over x [tokens][heads][elems] (the elements of a head
    contiguous) into `out` of the same shape, or in place.  positions: int32
    [tokens], turns: the table on the GPU; all must outlive the step."""
    out = x if out is None else out
    if x.dim() != 3 or out.shape != x.shape or out.dtype != x.dtype:
        raise ValueError("x and out: [tokens][heads][elems] of one type")
    if x.shape[2] > 1 and (x.stride(2) != 1 or out.stride(2) != 1):
        raise ValueError("the elements of a head must be contiguous")
    rotary = x.shape[2] - offset if rotary is None else rotary
    if _type_name(x.dtype) not in _WIDE:
        raise ValueError(f"a bfloat16 or float16 tensor is needed, not {x.dtype}")
    parts = _Parts()
    parts.reach(x, "x")
    parts.reach(out, "out")
    parts.entries(positions, "positions", ("int32",), x.shape[0])
    parts.entries(turns, "turns", _TURNS, rotary // 2)
    st = dhs_rotate_step()
    st.dtype = _DTYPES[_WIDE[_type_name(x.dtype)]]
    st.tokens, st.heads, st.head_elems = x.shape
    st.rotary_offset, st.rotary_elems, st.pairs = offset, rotary, _PAIRS[pairs]
    st.flags, st.amplitude = DHS_ROPE_INVERSE if inverse else 0, amplitude
    st.x_token_stride, st.x_head_stride = x.stride()[:2]
    st.y_token_stride, st.y_head_stride = out.stride()[:2]
    st.x_dev, st.y_dev = x.data_ptr(), out.data_ptr()
    st.position_dev, st.turns_dev = positions.data_ptr(), turns.data_ptr()
    return st


def dhs_rotate(h, st: dhs_rotate_step):
    return lib.dhs_rotate(h, ctypes.byref(st))


def dhs_rotate_on(h, st: dhs_rotate_step, stream):
    return lib.dhs_rotate_on(h, ctypes.byref(st), stream)


def packed_rows(*, key_elems, value_elems, kv_heads=1, wide_elems=0, shared=False,
                dtype="bf16") -> dhs_packed_rows:
    return dhs_packed_rows(_DTYPES[dtype], kv_heads, key_elems, wide_elems, value_elems, int(shared))


def dhs_packed_bytes(rows: dhs_packed_rows) -> int:
    n = _i32(0)
    check(lib.dhs_packed_bytes(ctypes.byref(rows), ctypes.byref(n)), "dhs_packed_bytes")
    return n.value


@functools.lru_cache(maxsize=64)
def _array_type(kind, n):
    return kind * n


def _array(kind, items):
    """The items as a C array; by their bytes, which is several times faster
    than an argument each."""
    if not items:
        return (kind * 1)()
    if set(map(type, items)) != {kind}:
        raise TypeError(f"{kind.__name__}s are needed")
    return _array_type(kind, len(items)).from_buffer_copy(b"".join(items))


# The items' fields: several times faster than a ctypes argument each.
_pack_pack_item, _pack_unpack_item = struct.Struct("=4i5Q").pack, struct.Struct("=3iIq4Q").pack
_new_pack_item, _new_unpack_item = dhs_pack_item.from_buffer_copy, dhs_unpack_item.from_buffer_copy


def pack_item(count, key, *, wide=None, value=None, positions=None, rows=None, req=0,
              src=0) -> dhs_pack_item:
    """A dhs_pack_item from torch tensors (or device addresses): key, wide and
    value of the layout's type, positions int32 [count], rows for dhs_pack the
    memory that packed rows go to."""
    it = _new_pack_item(_pack_pack_item(
        req, src, count, 0, 0 if key is None else _address(key), 0 if wide is None else _address(wide),
        0 if value is None else _address(value), 0 if positions is None else _address(positions),
        0 if rows is None else _address(rows)))
    it.given = count, key, wide, value, positions, rows  # for make_pack's checks
    return it


def make_pack(items, rows, *, rotary_offset=0, rotary_elems=0, pairs="half", amplitude=1.0,
              turns=None, key_strides=None, wide_strides=None, value_strides=None) -> tuple:
    """A dhs_pack_step plus the item array that must stay alive with it.
    Strides are (between tokens, between heads) in elements; the default is
    contiguous [count][kv_heads][elems].  ValueError for tensors of another type
    or with fewer elements, or that the GPU cannot reach."""
    arr = _array(dhs_pack_item, items)
    parts, n = _Parts(rows), rows.key_elems - rows.wide_elems
    for it in items:
        count, key, wide, value, positions, packed = getattr(it, "given", (0,) + 5 * (None,))
        if key is not None:
            parts.heads(key, "key", count, n, key_strides)
        if wide is not None and rows.wide_elems:
            parts.heads(wide, "wide", count, rows.wide_elems, wide_strides)
        if value is not None and not rows.shared:
            parts.heads(value, "value", count, rows.value_elems, value_strides)
        if rotary_elems:
            parts.entries(positions, "positions", ("int32",), count)
        if packed is not None:
            parts.packed(packed, count)
    if rotary_elems:
        parts.entries(turns, "turns", _TURNS, rotary_elems // 2)
    st = dhs_pack_step()
    st.rows, st.n_items, st.items = rows, len(items), arr
    st.rotary_offset, st.rotary_elems = rotary_offset, rotary_elems
    st.pairs, st.amplitude, st.turns_dev = _PAIRS[pairs], amplitude, _address(turns)
    flat = lambda m: (rows.kv_heads * m, m)  # noqa: E731
    st.key_token_stride, st.key_head_stride = key_strides or flat(n)
    st.wide_token_stride, st.wide_head_stride = wide_strides or flat(rows.wide_elems)
    st.value_token_stride, st.value_head_stride = value_strides or flat(rows.value_elems)
    return st, arr


def dhs_pack(h, st: dhs_pack_step):
    return lib.dhs_pack(h, ctypes.byref(st))


def dhs_append_packed(h, st: dhs_pack_step):
    return lib.dhs_append_packed(h, ctypes.byref(st))


def unpack_item(count, key, *, value=None, loc=None, rows=None, req=0, src=0, first=0,
                flags=0) -> dhs_unpack_item:
    """A dhs_unpack_item from torch tensors (or device addresses): key and value,
    of the layout's type, are written; loc is int32 [count], rows the memory that
    packed rows lie in."""
    it = _new_unpack_item(_pack_unpack_item(
        req, src, count, flags, first, 0 if loc is None else _address(loc),
        0 if rows is None else _address(rows), 0 if key is None else _address(key),
        0 if value is None else _address(value)))
    it.given = count, key, value, loc, rows  # for make_unpack's checks
    return it


def make_unpack(items, rows, *, key_strides=None, value_strides=None) -> tuple:
    """A dhs_unpack_step plus the item array that must stay alive with it.
    Strides are (between rows, between heads) in elements; the default is
    contiguous [count][kv_heads][elems].  ValueError for tensors of another type
    or with fewer elements, or that the GPU cannot reach."""
    arr = _array(dhs_unpack_item, items)
    parts, n, m, kv = _Parts(rows), rows.key_elems, rows.value_elems, rows.kv_heads
    device, dtype, flat = None, parts.dtype, key_strides is None
    for it in items:
        count, key, value, loc, packed = getattr(it, "given", (0,) + 4 * (None,))
        # a decode step's items differ in little: what heads() asks, without the call
        if key is not None and not (flat and device is not None and type(key) is kind and
                                    key.get_device() == device and key.dtype is dtype and
                                    key.numel() >= count * kv * n and key.is_contiguous()):
            parts.heads(key, "key", count, n, key_strides)
            device, kind = parts.device, type(key)
        if value is not None:
            parts.heads(value, "value", count, m, value_strides)
        if packed is not None and not it.flags & DHS_UNPACK_HISTORY:
            parts.packed(packed, count)
        elif loc is not None and not it.flags & DHS_UNPACK_HISTORY:
            parts.entries(loc, "loc", ("int32", "uint32"), count)
    st = dhs_unpack_step()
    st.rows, st.n_items, st.items = rows, len(items), arr
    st.key_row_stride, st.key_head_stride = key_strides or (kv * n, n)
    st.value_row_stride, st.value_head_stride = value_strides or (kv * m, m)
    return st, arr


def dhs_unpack(h, st: dhs_unpack_step):
    return lib.dhs_unpack(h, ctypes.byref(st))


def dhs_unpack_on(h, st: dhs_unpack_step, stream):
    return lib.dhs_unpack_on(h, ctypes.byref(st), stream)


def make_attend_packed(items, rows, *, heads, scale, q_strides=None, out_strides=None) -> tuple:
    """A dhs_attend_packed_step (without a workspace) over attend_item()s plus
    the item array that must stay alive with it; strides as make_attend's."""
    arr = _array(dhs_attend_item, items)
    st = dhs_attend_packed_step()
    st.rows, st.n_items, st.items, st.heads, st.scale = rows, len(items), arr, heads, scale
    n, m = rows.key_elems, rows.value_elems
    st.q_query_stride, st.q_head_stride = q_strides or (heads * n, n)
    st.out_query_stride, st.out_head_stride = out_strides or (heads * m, m)
    return st, arr


def dhs_attend_packed_bytes(h, st: dhs_attend_packed_step) -> int:
    n = ctypes.c_size_t(0)
    check(lib.dhs_attend_packed_bytes(h, ctypes.byref(st), ctypes.byref(n)),
          "dhs_attend_packed_bytes")
    return n.value


def dhs_attend_packed(h, st: dhs_attend_packed_step):
    return lib.dhs_attend_packed(h, ctypes.byref(st))


def dhs_attend_packed_on(h, st: dhs_attend_packed_step, stream):
    return lib.dhs_attend_packed_on(h, ctypes.byref(st), stream)


def dhs_fork(h, req, child, host_ptrs, masks=None):
    """host_ptrs: one pinned address per source (0: none); masks: None, or one
    resident-page mask or None per source."""
    hosts = (_vp * max(1, len(host_ptrs)))(*host_ptrs)
    keep, mp = [], None
    if masks is not None:
        keep = [None if m is None else np.ascontiguousarray(m, np.uint8) for m in masks]
        mp = (_vp * max(1, len(keep)))(*[None if m is None else m.ctypes.data for m in keep])
    d = _i64(0)
    rc = lib.dhs_fork(h, req, child, hosts, mp, ctypes.byref(d))
    return rc, d.value


def dhs_compact(h, capacity_pages):
    n = _i64(0)
    rc = lib.dhs_compact(h, capacity_pages, ctypes.byref(n))
    return rc, n.value


def dhs_resolve(h, st: dhs_step):
    return lib.dhs_resolve(h, ctypes.byref(st))


def dhs_gather(h, st: dhs_step):
    return lib.dhs_gather(h, ctypes.byref(st))


def dhs_resolve_gather(h, st: dhs_step):
    return lib.dhs_resolve_gather(h, ctypes.byref(st))


def dhs_decode_step(h, appends, st: dhs_step):
    arr = (dhs_append_item * max(1, len(appends)))(*appends)
    return lib.dhs_decode_step(h, arr, len(appends), ctypes.byref(st))


def dhs_status(h):
    f = _u32(0)
    rc = lib.dhs_status(h, ctypes.byref(f))
    return rc, f.value


def dhs_set_option(h, key, value):
    return lib.dhs_set_option(h, key, value)


def dhs_get_option(h, key):
    v = _i64(0)
    rc = lib.dhs_get_option(h, key, ctypes.byref(v))
    return rc, v.value


def dhs_read_state(h, req, src, B, pages_max):
    tags = np.empty(B, np.int32)
    stamps = np.empty(B, np.uint32)
    pages = np.empty(pages_max, np.int32)
    info = np.empty(4, np.int64)
    check(lib.dhs_read_state(h, req, src, tags.ctypes.data, stamps.ctypes.data,
                             pages.ctypes.data, info.ctypes.data), "dhs_read_state")
    return tags, stamps, pages, info


# ------------------------------------------------------------ host memory

class HostRows:
    """Page-aligned host memory registered as mapped pinned memory.

    ``array`` is a uint8 numpy view; ``ptr`` is the host address the library
    receives (it derives the device-visible address itself).
    """

    def __init__(self, nbytes: int, hugepages: bool = True):
        import torch
        self.nbytes = max(int(nbytes), 4096)
        self._mm = mmap.mmap(-1, self.nbytes)
        if hugepages and hasattr(mmap, "MADV_HUGEPAGE"):
            # ask for transparent huge pages (the GPU reads missing rows from
            # this memory at random offsets); where the kernel grants none the
            # advice changes nothing
            try:
                self._mm.madvise(mmap.MADV_HUGEPAGE)
            except OSError:
                pass
        self.array = np.frombuffer(self._mm, dtype=np.uint8)
        self.ptr = self.array.ctypes.data
        rc = torch._C._cudart.cudaHostRegister(self.ptr, self.nbytes, 3)  # portable|mapped
        if int(rc) != 0:
            raise RuntimeError(f"cudaHostRegister failed: {rc}")
        self._registered = True

    def close(self):
        if getattr(self, "_registered", False):
            import torch
            torch._C._cudart.cudaHostUnregister(self.ptr)
            self._registered = False
        self.array = None
        if getattr(self, "_mm", None) is not None:
            try:
                self._mm.close()
            except BufferError:
                pass
            self._mm = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Pool:
    """A dhs pool with its four device arenas allocated by torch, or with the
    caller's own hot, tail and optional arenas (`arenas`, contiguous uint8
    tensors of dhs_pool_bytes' sizes).  A caller's hot arena must not hold
    rows the pool should know: a pool starts with empty hot caches."""

    def __init__(self, *, max_requests, sources, row_bytes, page_rows, tail_rows,
                 hot_rows, max_queries, max_topk, max_rows_per_request,
                 optional_pages, admission_reserve_pages=0, device=None,
                 stream=None, arenas=None):
        import torch
        self.device = torch.device(device or "cuda")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.stream = stream or torch.cuda.current_stream(self.device)
        cfg = dhs_pool_config()
        cfg.max_requests, cfg.sources, cfg.row_bytes = max_requests, sources, row_bytes
        cfg.page_rows, cfg.tail_rows, cfg.hot_rows = page_rows, tail_rows, hot_rows
        cfg.max_queries, cfg.max_topk = max_queries, max_topk
        cfg.max_rows_per_request = max_rows_per_request
        cfg.optional_pages = optional_pages
        cfg.admission_reserve_pages = admission_reserve_pages
        sizes = dhs_pool_bytes(cfg)
        given = list(arenas or ())
        for a, s in zip(given, sizes):
            if a.dtype != torch.uint8 or not a.is_contiguous() or a.numel() < s:
                raise ValueError(f"an arena of {s} contiguous bytes is needed")
            if a.device != self.device:
                raise ValueError(f"an arena on {self.device} is needed, not on {a.device}")
        self.buffers = given + [torch.empty(max(s, 256), dtype=torch.uint8, device=self.device)
                                for s in sizes[len(given):]]
        cfg.hot_dev, cfg.tail_dev, cfg.opt_dev, cfg.meta_dev = [
            b.data_ptr() for b in self.buffers]
        cfg.stream = self.stream.cuda_stream
        self.cfg = cfg
        self.pages_max = -(-max_rows_per_request // page_rows)
        with torch.cuda.device(self.device):
            self.h = dhs_pool_create(cfg)

    @property
    def hot(self):
        return self.buffers[DHS_BUF_HOT]

    @property
    def tail(self):
        return self.buffers[DHS_BUF_TAIL]

    @property
    def opt(self):
        return self.buffers[DHS_BUF_OPT]

    def close(self):
        if getattr(self, "h", None):
            self.stream.synchronize()
            dhs_pool_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def admit(self, req, src, host_ptr, n_rows, mask=None):
        return dhs_admit(self.h, req, src, host_ptr, n_rows, mask)

    def reclaim(self, order, deficit):
        return dhs_reclaim(self.h, order, deficit)

    def release(self, req):
        return dhs_release(self.h, req)

    def admit_device(self, req, src, dev_ptr, host_ptr, n_rows, mask=None):
        return dhs_admit_device(self.h, req, src, dev_ptr, host_ptr, n_rows, mask)

    def admit_window(self, req, src, dev_ptr, n_rows):
        return dhs_admit_window(self.h, req, src, dev_ptr, n_rows)

    def backup(self, max_pages):
        return dhs_backup(self.h, max_pages)

    def refill(self, max_pages):
        return dhs_refill(self.h, max_pages)

    def pending_backup(self):
        return int(lib.dhs_pending_backup(self.h))

    def used(self):
        return dhs_pool_used(self.h)

    def flush(self):
        return dhs_flush(self.h)

    def append(self, items):
        return dhs_append(self.h, items)

    def resolve(self, st):
        return dhs_resolve(self.h, st)

    def gather(self, st):
        return dhs_gather(self.h, st)

    def resolve_gather(self, st):
        return dhs_resolve_gather(self.h, st)

    def attend_bytes(self, st):
        return dhs_attend_bytes(self.h, st)

    def attend(self, st):
        return dhs_attend(self.h, st)

    def attend_on(self, st, stream):
        return dhs_attend_on(self.h, st, stream)

    def rotate(self, st):
        return dhs_rotate(self.h, st)

    def rotate_on(self, st, stream):
        return dhs_rotate_on(self.h, st, stream)

    def pack(self, st):
        return dhs_pack(self.h, st)

    def append_packed(self, st):
        return lib.dhs_append_packed(self.h, ctypes.byref(st))

    def unpack(self, st):
        return lib.dhs_unpack(self.h, ctypes.byref(st))

    def unpack_on(self, st, stream):
        return dhs_unpack_on(self.h, st, stream)

    def attend_packed_bytes(self, st):
        return dhs_attend_packed_bytes(self.h, st)

    def attend_packed(self, st):
        return dhs_attend_packed(self.h, st)

    def attend_packed_on(self, st, stream):
        return dhs_attend_packed_on(self.h, st, stream)

    def fork(self, req, child, host_ptrs, masks=None):
        return dhs_fork(self.h, req, child, host_ptrs, masks)

    def compact(self, capacity_pages):
        return dhs_compact(self.h, capacity_pages)

    def capacity(self):
        return int(lib.dhs_pool_capacity(self.h))

    def status(self):
        return dhs_status(self.h)

    def set_option(self, key, value):
        return check(dhs_set_option(self.h, key, value), "dhs_set_option")

    def get_option(self, key):
        rc, v = dhs_get_option(self.h, key)
        check(rc, "dhs_get_option")
        return v

    def read_state(self, req, src):
        return dhs_read_state(self.h, req, src, self.cfg.hot_rows, self.pages_max)
