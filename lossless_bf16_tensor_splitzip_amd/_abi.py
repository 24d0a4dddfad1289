"""ctypes binding of the C ABI in include/splitzip.h and include/splitzip_kv.h.

Argument marshalling only: every step of calibrate / encode / decode runs in
the HIP kernels of ``_lib/libsplitzip.so``, every step of the key-value cache
in those of ``_lib/libsplitzip_kv.so``.  They must have been built
(``python -m lossless_bf16_tensor_splitzip_amd._build`` or
``__graft_entry__.build()``); there is no fallback of any kind.
"""
from __future__ import annotations

import ctypes
import os

from ._build import CEILING_LIB_PATH, KV_LIB_PATH, LIB_PATH

CHUNK = 1024
MAX_N = 1 << 36
NOALLOC_MAX_N = 133627904        # splitzip_encode_noalloc's limit

OK = 0
ERR_INVALID = 1
ERR_CAPACITY = 2
ERR_CORRUPT = 3
ERR_HIP = 4
ERR_WORKSPACE = 5
ERR_INTERNAL = 6

# splitzip_meta.flags
META_ASCENDING = 1

# decode status bits
DEC_BAD_META = 1
DEC_ESC_OUT_OF_RANGE = 2
DEC_POS_GE_CHUNK = 4
DEC_NOT_INCREASING = 8


class Codebook(ctypes.Structure):
    """Mirror of splitzip_codebook."""
    _fields_ = [
        ("enc_lut", ctypes.c_uint8 * 256),
        ("enc_lut_marked", ctypes.c_uint8 * 256),
        ("dec_lut", ctypes.c_uint8 * 16),
        ("common_lut", ctypes.c_uint8 * 256),
        ("n_codes", ctypes.c_uint32),
        ("reserved", ctypes.c_uint32),
        ("covered", ctypes.c_uint64),
        ("total", ctypes.c_uint64),
        ("counts", ctypes.c_uint64 * 256),
    ]


class Meta(ctypes.Structure):
    """Mirror of splitzip_meta."""
    _fields_ = [
        ("n", ctypes.c_uint64),
        ("n_pairs", ctypes.c_uint64),
        ("chunk_size", ctypes.c_uint64),
        ("n_esc", ctypes.c_uint64),
        ("comp_bytes", ctypes.c_uint64),
        ("offsets", ctypes.c_uint64 * 5),
        ("covered", ctypes.c_uint64),
        ("total", ctypes.c_uint64),
        ("status", ctypes.c_int32),
        ("flags", ctypes.c_uint32),
    ]


class Item(ctypes.Structure):
    """Mirror of splitzip_item (one tensor of a batched call; device pointers)."""
    _fields_ = [
        ("x", ctypes.c_void_p),
        ("n", ctypes.c_uint64),
        ("cb", ctypes.c_void_p),
        ("payload", ctypes.c_void_p),
        ("capacity", ctypes.c_uint64),
        ("meta", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
    ]


class SlotItem(ctypes.Structure):
    """Mirror of splitzip_slot_item (one payload of a batched in-place decode)."""
    _fields_ = [
        ("slot", ctypes.c_void_p),
        ("slot_bytes", ctypes.c_uint64),
        ("meta", ctypes.c_void_p),
        ("dec_lut", ctypes.c_void_p),
        ("n", ctypes.c_uint64),
        ("stash", ctypes.c_void_p),
        ("stash_bytes", ctypes.c_uint64),
    ]


DEC_LUT_OFFSET = Codebook.dec_lut.offset

# name -> (restype, argtypes), exactly the functions of include/splitzip.h
_P = ctypes.c_void_p
_U64 = ctypes.c_uint64
_SZ = ctypes.c_size_t
SIGNATURES = {
    "splitzip_abi_version": (ctypes.c_int, []),
    "splitzip_struct_sizes": (None, [ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t)]),
    "splitzip_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "splitzip_payload_size": (_U64, [_U64, _U64]),
    "splitzip_slot_schedule": (ctypes.c_uint32, [_U64, ctypes.c_uint32, ctypes.POINTER(_U64),
                                                ctypes.POINTER(_U64), ctypes.POINTER(_U64)]),
    "splitzip_workspace_size": (_SZ, [_U64]),
    "splitzip_workspace_init": (ctypes.c_int, [_P, _SZ, _P]),
    "splitzip_calibrate": (ctypes.c_int, [_P, _U64, _P, _P, _SZ, _P]),
    "splitzip_encode": (ctypes.c_int, [_P, _U64, _P, _P, _U64, _P, _P, _SZ, _P]),
    "splitzip_encode_chunked": (ctypes.c_int, [_P, _U64, _P, ctypes.c_uint32, _P, _U64, _P, _P, _SZ,
                                               _P]),
    "splitzip_encode_noalloc": (ctypes.c_int, [_P, _U64, _P, _P, _U64, _P, _P]),
    "splitzip_decode": (ctypes.c_int, [_P, _U64, _P, _P, _P, _U64, _P, _P]),
    "splitzip_decode_slot": (ctypes.c_int, [_P, _U64, _P, _P, _U64, _P, _U64, _P, _P]),
    "splitzip_decode_slot_batch": (ctypes.c_int, [_P, ctypes.c_uint32, _P, _P]),
    "splitzip_decode_slot_batch_resident": (ctypes.c_int, [_P, ctypes.c_uint32, _P, _P]),
    "splitzip_workspace_size_batch": (_SZ, [ctypes.POINTER(ctypes.c_uint64), ctypes.c_uint32]),
    "splitzip_calibrate_batch": (ctypes.c_int, [_P, ctypes.c_uint32, _P, _SZ, _P]),
    "splitzip_encode_batch": (ctypes.c_int, [_P, ctypes.c_uint32, _P, _SZ, _P]),
    "splitzip_decode_batch": (ctypes.c_int, [_P, ctypes.c_uint32, _P, _P]),
}

_lib = None


CEILING_SIGNATURES = {
    "splitzip_ceiling_read": (ctypes.c_int, [_P, ctypes.c_uint64, ctypes.c_uint32, _P, _P]),
    "splitzip_ceiling_encode_shape": (ctypes.c_int, [_P, ctypes.c_uint64, _P, _P, _P]),
    "splitzip_ceiling_decode_shape": (ctypes.c_int, [_P, _P, _P, ctypes.c_uint64, _P]),
    "splitzip_ceiling_order": (ctypes.c_int, [ctypes.c_uint32, ctypes.c_uint32, _P, _P, _P, _P,
                                              ctypes.c_uint64, _P]),
    "splitzip_ceiling_encode_wide": (ctypes.c_int, [_P, ctypes.c_uint64, _P, _P, _P]),
    "splitzip_ceiling_decode_wide": (ctypes.c_int, [_P, _P, _P, ctypes.c_uint64, _P]),
    "splitzip_ceiling_encode_arrive": (ctypes.c_int, [_P, ctypes.c_uint64, _P, _P, _P, _P, _P,
                                                      ctypes.c_uint32, _P]),
    "splitzip_ceiling_encode_fenced": (ctypes.c_int, [_P, ctypes.c_uint64, _P, _P, _P]),
    "splitzip_ceiling_atomics": (ctypes.c_int, [_P, ctypes.c_uint32, ctypes.c_uint32,
                                                ctypes.c_uint32, _P]),
    "splitzip_ceiling_launch": (ctypes.c_int, [ctypes.c_uint32, ctypes.c_uint32, _P, _P]),
}

_ceiling = None


def ceiling_lib():
    """Load the reference-stream library (measurement only; raises if it has
    not been built)."""
    global _ceiling
    if _ceiling is not None:
        return _ceiling
    if not os.path.exists(CEILING_LIB_PATH):
        raise RuntimeError("reference-stream library not built (%s missing)" % CEILING_LIB_PATH)
    handle = ctypes.CDLL(CEILING_LIB_PATH)
    for name, (res, args) in CEILING_SIGNATURES.items():
        fn = getattr(handle, name)
        fn.restype = res
        fn.argtypes = args
    _ceiling = handle
    return handle


# include/splitzip_kv.h (strides as single fields: the same layout as the
# header's arrays, cheaper to fill)

KV_BF16 = 0
KV_FP16 = 1
KV_ALL = 0xFFFFFFFF

# status bits of the key-value cache calls
KV_BAD_PAGE = 1
KV_BAD_LEN = 2
KV_BAD_ROWS = 4
KV_NO_PAGE = 8
KV_BAD_PARENT = 16
KV_MAX_PAGES = 1 << 24
KV_MAX_LAYERS = 1024
KV_MAX_GROUPS = 65535

_U32 = ctypes.c_uint32


class KVCacheArgs(ctypes.Structure):
    """Mirror of splitzip_kv_cache."""
    _fields_ = [
        ("k", _P), ("v", _P),
        ("k_stride0", _U64), ("k_stride1", _U64), ("k_stride2", _U64),
        ("v_stride0", _U64), ("v_stride1", _U64), ("v_stride2", _U64),
        ("table", _P), ("table_stride", _U64), ("lens", _P),
        ("num_pages", _U32), ("page_size", _U32), ("kv_heads", _U32), ("head_dim", _U32),
        ("batch", _U32), ("max_pages", _U32), ("dtype", _U32), ("reserved", _U32),
    ]


class KVRows(ctypes.Structure):
    """Mirror of splitzip_kv_rows."""
    _fields_ = [
        ("k", _P), ("v", _P),
        ("k_stride0", _U64), ("k_stride1", _U64), ("v_stride0", _U64), ("v_stride1", _U64),
        ("rows", _U32), ("reserved", _U32), ("cu", _P), ("start", _P),
    ]


class KVQuery(ctypes.Structure):
    """Mirror of splitzip_kv_query."""
    _fields_ = [
        ("q", _P), ("q_stride0", _U64), ("q_stride1", _U64),
        ("out", _P), ("out_stride0", _U64), ("out_stride1", _U64),
        ("lse", _P), ("mass", _P), ("mass_out", _P),
        ("mass_stride0", _U64), ("mass_stride1", _U64),
        ("mass_out_stride0", _U64), ("mass_out_stride1", _U64),
        ("heads", _U32), ("window", _U32), ("sinks", _U32), ("scale", ctypes.c_float),
        ("mass_len", _U32), ("reserved", _U32),
    ]


class KVBudget(ctypes.Structure):
    """Mirror of splitzip_kv_budget."""
    _fields_ = [
        ("mass", _P), ("mass_out", _P),
        ("mass_stride0", _U64), ("mass_stride1", _U64),
        ("mass_out_stride0", _U64), ("mass_out_stride1", _U64),
        ("kept", _P), ("budget", _U32), ("sinks", _U32), ("recent", _U32), ("mass_len", _U32),
    ]


class KVGroups(ctypes.Structure):
    """Mirror of splitzip_kv_groups."""
    _fields_ = [("cu", _P), ("shared", _P), ("groups", _U32), ("reserved", _U32)]


class KVPagesArgs(ctypes.Structure):
    """Mirror of splitzip_kv_pages."""
    _fields_ = [
        ("cache", _P), ("k", _P), ("v", _P), ("layers", _U32), ("reserved", _U32),
        ("state", _P), ("state_bytes", _SZ),
    ]


KV_STRUCTS = (KVCacheArgs, KVRows, KVQuery, KVBudget)

KV_SIGNATURES = {
    "splitzip_kv_struct_sizes": (None, [ctypes.POINTER(ctypes.c_size_t)]),
    "splitzip_kv_append": (ctypes.c_int, [_P, _P, _P, _P]),
    "splitzip_kv_gather": (ctypes.c_int, [_P, _P, _P, _P]),
    "splitzip_kv_attend_workspace_size": (_SZ, [_P, _U32, _U32]),
    "splitzip_kv_attend": (ctypes.c_int, [_P, _P, _P, _SZ, _P, _P]),
    "splitzip_kv_evict": (ctypes.c_int, [_P, _P, _P, _P, _P]),
    "splitzip_kv_groups_struct_size": (_SZ, []),
    "splitzip_kv_shared_workspace_size": (_SZ, [_P, _U32, _U32]),
    "splitzip_kv_attend_shared": (ctypes.c_int, [_P, _P, _P, _P, _SZ, _P, _P]),
    "splitzip_kv_pages_struct_size": (_SZ, []),
    "splitzip_kv_pages_state_size": (_SZ, [_P]),
    "splitzip_kv_pages_count": (ctypes.c_int, [_P, _P, _P]),
    "splitzip_kv_pages_fork": (ctypes.c_int, [_P, _P, _P, _P]),
    "splitzip_kv_pages_resize": (ctypes.c_int, [_P, _P, _P, _P]),
    "splitzip_kv_pages_compact": (ctypes.c_int, [_P, _P, _P, _P, _P]),
    "splitzip_kv_pages_copy": (ctypes.c_int, [_P, _P, _P, _P, _U32, _P, _P]),
}

_kv = None


def kv_lib():
    """Load the key-value cache library (raises if it has not been built)."""
    global _kv
    if _kv is not None:
        return _kv
    if not os.path.exists(KV_LIB_PATH):
        raise RuntimeError(
            "SplitZip key-value cache library not built (%s missing): run "
            "`python -m lossless_bf16_tensor_splitzip_amd._build`" % KV_LIB_PATH)
    handle = ctypes.CDLL(KV_LIB_PATH)
    for name, (res, args) in KV_SIGNATURES.items():
        fn = getattr(handle, name)
        fn.restype = res
        fn.argtypes = args
    sizes = (ctypes.c_size_t * len(KV_STRUCTS))()
    handle.splitzip_kv_struct_sizes(sizes)
    if list(sizes) != [ctypes.sizeof(t) for t in KV_STRUCTS] or \
            handle.splitzip_kv_groups_struct_size() != ctypes.sizeof(KVGroups) or \
            handle.splitzip_kv_pages_struct_size() != ctypes.sizeof(KVPagesArgs):
        raise RuntimeError("struct layout mismatch between the library and the binding")
    _kv = handle
    return handle


def lib():
    """Load the HIP library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            "SplitZip HIP library not built (%s missing): run "
            "`python -m lossless_bf16_tensor_splitzip_amd._build`" % LIB_PATH)
    handle = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(handle, name)
        fn.restype = res
        fn.argtypes = args
    cb_size, meta_size = ctypes.c_size_t(), ctypes.c_size_t()
    handle.splitzip_struct_sizes(ctypes.byref(cb_size), ctypes.byref(meta_size))
    if cb_size.value != ctypes.sizeof(Codebook) or meta_size.value != ctypes.sizeof(Meta):
        raise RuntimeError("struct layout mismatch between the library and the binding")
    _lib = handle
    return handle


class SplitZipError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__("%s failed: %s (%d)" % (fn, status_string(status), status))


def status_string(status: int) -> str:
    return lib().splitzip_status_string(status).decode()


def _check(fn: str, status: int) -> int:
    if status != OK:
        raise SplitZipError(fn, status)
    return status


# Thin wrappers with the C names (raw pointers / ints in, status out).

def splitzip_abi_version() -> int:
    return lib().splitzip_abi_version()


def splitzip_payload_size(n: int, n_esc: int) -> int:
    return lib().splitzip_payload_size(n, n_esc)


def splitzip_slot_schedule(n: int, passes: int):
    """(passes used, t_min, lo, hi) of the in-place decode's pass schedule;
    lo and hi are lists of passes + 1 entries.  None for invalid arguments."""
    t_min = ctypes.c_uint64()
    lo = (ctypes.c_uint64 * (passes + 1))()
    hi = (ctypes.c_uint64 * (passes + 1))()
    used = lib().splitzip_slot_schedule(n, passes, ctypes.byref(t_min), lo, hi)
    if used == 0:
        return None
    return used, t_min.value, list(lo), list(hi)


def splitzip_workspace_size(n: int) -> int:
    return lib().splitzip_workspace_size(n)


def splitzip_workspace_init(d_ws: int, ws_bytes: int, stream: int) -> int:
    return lib().splitzip_workspace_init(d_ws, ws_bytes, stream)


def splitzip_calibrate(d_x: int, n: int, d_cb: int, d_ws: int, ws_bytes: int, stream: int) -> int:
    return lib().splitzip_calibrate(d_x, n, d_cb, d_ws, ws_bytes, stream)


def splitzip_encode(d_x: int, n: int, d_cb: int, d_payload: int, capacity: int, d_meta: int,
                    d_ws: int, ws_bytes: int, stream: int) -> int:
    return lib().splitzip_encode(d_x, n, d_cb, d_payload, capacity, d_meta, d_ws, ws_bytes, stream)


def splitzip_encode_chunked(d_x: int, n: int, d_cb: int, chunk_size: int, d_payload: int,
                            capacity: int, d_meta: int, d_ws: int, ws_bytes: int,
                            stream: int) -> int:
    return lib().splitzip_encode_chunked(d_x, n, d_cb, chunk_size, d_payload, capacity, d_meta,
                                         d_ws, ws_bytes, stream)


def splitzip_encode_noalloc(d_x: int, n: int, d_cb: int, d_payload: int, capacity: int,
                            d_meta: int, stream: int) -> int:
    return lib().splitzip_encode_noalloc(d_x, n, d_cb, d_payload, capacity, d_meta, stream)


def splitzip_decode(d_payload: int, payload_bytes: int, d_meta: int, d_dec_lut: int, d_out: int,
                    n: int, d_status: int, stream: int) -> int:
    return lib().splitzip_decode(d_payload, payload_bytes, d_meta, d_dec_lut, d_out, n, d_status,
                                 stream)


def splitzip_decode_slot(d_slot: int, slot_bytes: int, d_meta: int, d_dec_lut: int, n: int,
                         d_stash: int, stash_bytes: int, d_status: int, stream: int) -> int:
    return lib().splitzip_decode_slot(d_slot, slot_bytes, d_meta, d_dec_lut, n, d_stash,
                                      stash_bytes, d_status, stream)


def splitzip_decode_slot_batch(items, count: int, d_status: int, stream: int) -> int:
    return lib().splitzip_decode_slot_batch(_items_ptr(items), count, d_status, stream)


def splitzip_decode_slot_batch_resident(items, count: int, d_status: int, stream: int) -> int:
    return lib().splitzip_decode_slot_batch_resident(_items_ptr(items), count, d_status, stream)


def splitzip_workspace_size_batch(ns) -> int:
    arr = (ctypes.c_uint64 * max(len(ns), 1))(*ns)
    return lib().splitzip_workspace_size_batch(arr, len(ns))


def _items_ptr(items):
    return ctypes.cast(items, ctypes.c_void_p) if items is not None else None


def splitzip_calibrate_batch(items, count: int, d_ws: int, ws_bytes: int, stream: int) -> int:
    return lib().splitzip_calibrate_batch(_items_ptr(items), count, d_ws, ws_bytes, stream)


def splitzip_encode_batch(items, count: int, d_ws: int, ws_bytes: int, stream: int) -> int:
    return lib().splitzip_encode_batch(_items_ptr(items), count, d_ws, ws_bytes, stream)


def splitzip_decode_batch(items, count: int, d_status: int, stream: int) -> int:
    return lib().splitzip_decode_batch(_items_ptr(items), count, d_status, stream)


# Key-value cache (structs by reference, raw pointers / ints in, status out).

def splitzip_kv_append(cache, rows, d_status: int, stream: int) -> int:
    return kv_lib().splitzip_kv_append(ctypes.byref(cache), ctypes.byref(rows), d_status, stream)


def splitzip_kv_gather(cache, rows, d_status: int, stream: int) -> int:
    return kv_lib().splitzip_kv_gather(ctypes.byref(cache), ctypes.byref(rows), d_status, stream)


def splitzip_kv_attend_workspace_size(cache, heads: int, mass_len: int) -> int:
    return kv_lib().splitzip_kv_attend_workspace_size(ctypes.byref(cache), heads, mass_len)


def splitzip_kv_attend(cache, query, d_ws: int, ws_bytes: int, d_status: int, stream: int) -> int:
    return kv_lib().splitzip_kv_attend(ctypes.byref(cache), ctypes.byref(query), d_ws, ws_bytes,
                                       d_status, stream)


def splitzip_kv_evict(cache, to, budget, d_status: int, stream: int) -> int:
    return kv_lib().splitzip_kv_evict(ctypes.byref(cache), ctypes.byref(to), ctypes.byref(budget),
                                      d_status, stream)


def splitzip_kv_groups_struct_size() -> int:
    return kv_lib().splitzip_kv_groups_struct_size()


def splitzip_kv_shared_workspace_size(cache, heads: int, groups: int) -> int:
    return kv_lib().splitzip_kv_shared_workspace_size(ctypes.byref(cache), heads, groups)


def splitzip_kv_attend_shared(cache, query, groups, d_ws: int, ws_bytes: int, d_status: int, stream: int) -> int:
    return kv_lib().splitzip_kv_attend_shared(ctypes.byref(cache), ctypes.byref(query), ctypes.byref(groups), d_ws, ws_bytes,
                                              d_status, stream)


def splitzip_kv_pages_struct_size() -> int:
    return kv_lib().splitzip_kv_pages_struct_size()


def splitzip_kv_pages_state_size(cache) -> int:
    return kv_lib().splitzip_kv_pages_state_size(ctypes.byref(cache))


def splitzip_kv_pages_count(pages, d_status: int, stream: int) -> int:
    return kv_lib().splitzip_kv_pages_count(ctypes.byref(pages), d_status, stream)


def splitzip_kv_pages_fork(pages, parents: int, d_status: int, stream: int) -> int:
    return kv_lib().splitzip_kv_pages_fork(ctypes.byref(pages), parents, d_status, stream)


def splitzip_kv_pages_resize(pages, lens: int, d_status: int, stream: int) -> int:
    return kv_lib().splitzip_kv_pages_resize(ctypes.byref(pages), lens, d_status, stream)


def splitzip_kv_pages_compact(pages, moved: int, used: int, d_status: int, stream: int) -> int:
    return kv_lib().splitzip_kv_pages_compact(ctypes.byref(pages), moved, used, d_status, stream)


def splitzip_kv_pages_copy(from_pages, to_pages, src: int, dst: int, n: int, d_status: int, stream: int) -> int:
    return kv_lib().splitzip_kv_pages_copy(ctypes.byref(from_pages), ctypes.byref(to_pages), src, dst, n, d_status,
                                           stream)
