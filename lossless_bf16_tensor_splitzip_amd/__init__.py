"""SplitZip lossless BF16 codec for MI355X (gfx950).

Hand-written HIP kernels behind the C ABI of include/splitzip.h
(``_lib/libsplitzip.so``); this package is the thin Python binding:

* ``_abi``   -- ctypes view of the C functions (same names) and structs;
* ``codec``  -- torch-tensor marshalling: Workspace, calibrate, encode, decode;
* ``persist`` -- codebook / metadata JSON and the 0.99 coverage gate;
* ``kv``      -- the paged key-value cache that decoded tensors go into:
  append, gather, attention of one new token (also over sequences that begin
  alike), eviction
  (``_lib/libsplitzip_kv.so``, include/splitzip_kv.h);
* ``kv_pages`` -- who has which of its pages: counting, forking, resizing,
  compacting, copying.

The method: page "splitzip_codec.py -- SplitZip codec adapter for
diffusers-dynamic-offloader" and page "SplitZip in DDO -- VMM routes".
"""
from ._abi import CHUNK, Codebook, Meta, SplitZipError, lib  # noqa: F401
from . import persist  # noqa: F401
from .codec import (Batch, Workspace, calibrate, decode, decode_slot, decode_slots,  # noqa: F401
                    encode, payload_for, payload_size, read_codebook, read_meta)
from .kv import KVCache, KVSharedWorkspace, KVWorkspace  # noqa: F401
from .kv_pages import KVPages  # noqa: F401

__all__ = ["CHUNK", "Batch", "Codebook", "KVCache", "KVPages", "KVSharedWorkspace", "KVWorkspace", "Meta", "SplitZipError", "Workspace", "calibrate", "encode",
           "decode", "decode_slot", "decode_slots", "payload_for", "payload_size", "read_codebook", "read_meta",
           "lib", "persist"]
