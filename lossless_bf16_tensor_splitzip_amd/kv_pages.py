"""Who has which pages of a paged key-value cache: marshalling of torch tensors
into the page operators of include/splitzip_kv.h.  All of it happens on the
device, in the HIP kernels; nothing is read back.

    pages = KVPages([cache of each layer])      # one table, one lens
    pages.count()                               # once: who has what
    pages.resize(new_lens)                      # a step: room for its tokens, each sequence's own
    cache.append(k, v, cu)                      # of each layer
    pages.fork(parents)                         # sequences continue others; -1 frees one
    pages.compact()                             # the pages in use to the front of the pools
"""
from __future__ import annotations

import ctypes

import torch

from . import _abi
from .kv import KVCache, _meet, _raw_stream, _span

_SHARED = ("batch", "max_pages", "kv_heads", "page_size", "head_dim", "dtype", "device")


class KVPages:
    """The pages of one cache, or of the caches of a model's layers, which have
    one table and one lens tensor, and pools of one shape and strides that
    share no memory.  It keeps how many table entries name each page, ``refs``
    (int32 [pages], to be read only): a page that none names is free.  Table
    and lengths are the caller's to read; pages are taken and given back by the
    calls below, one after another on one stream (or ordered by events).

    ``stream`` and ``status`` are as for ``KVCache``; further bits are
    _abi.KV_NO_PAGE (no page left: a sequence is shorter than asked for) and
    KV_BAD_PARENT (a parent outside the batch: the sequence is left)."""

    def __init__(self, caches: "KVCache | list[KVCache]"):
        caches = [caches] if isinstance(caches, KVCache) else list(caches)
        if not 1 <= len(caches) <= _abi.KV_MAX_LAYERS:
            raise ValueError("pages of 1 to %d layers, got %d" % (_abi.KV_MAX_LAYERS, len(caches)))
        first, a = caches[0], caches[0].args
        for c in caches[1:]:
            b = c.args
            if any(getattr(c, k) != getattr(first, k) for k in _SHARED) or a.num_pages != b.num_pages or \
                    any(getattr(a, k) != getattr(b, k) for k, _ in a._fields_ if k.startswith(("k_stride", "v_stride"))):
                raise ValueError("the layers' caches differ in shape, strides, dtype or device")
            if (a.table, a.table_stride, a.lens) != (b.table, b.table_stride, b.lens):
                raise ValueError("the layers' caches must have one table and one lens tensor")
        if a.num_pages > _abi.KV_MAX_PAGES or first.page_size * first.kv_heads * first.head_dim >> 34:
            raise ValueError("at most %d pages, each below 32 GiB" % _abi.KV_MAX_PAGES)
        if first.batch * first.max_pages >> 31:
            raise ValueError("a table of 2^31 entries")
        self.caches, self.device = caches, first.device
        self._apart_pools()
        self._kind = tuple(getattr(first, k) for k in _SHARED[2:])
        nbytes = _abi.splitzip_kv_pages_state_size(a)
        self.state = self._buffer(nbytes, self.device)
        self.refs = self.state.view(torch.int32)[:a.num_pages]
        layers = len(caches)
        self._k = (ctypes.c_void_p * layers)(*[c.args.k for c in caches])
        self._v = (ctypes.c_void_p * layers)(*[c.args.v for c in caches])
        self.args = _abi.KVPagesArgs(ctypes.addressof(a), ctypes.addressof(self._k), ctypes.addressof(self._v), layers, 0,
                                     self.state.data_ptr(), nbytes)
        self._ref, self._index, self._counted = ctypes.byref(self.args), self.device.index, False
        self._written = [_span(t) for t in (first.table, first.lens, self.state)]

    def _buffer(self, nbytes: int, device) -> torch.Tensor:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)

    def _apart_pools(self) -> None:
        """Notes where the pools lie, by their starts, and refuses some that meet."""
        pools = [(_span(t), (layer, name), t) for layer, c in enumerate(self.caches)
                 for name, t in (("k", c.k_pages), ("v", c.v_pages))]
        self._pools = sorted(pools, key=lambda x: x[0])
        self._reach = self._pools[0][0][0], max(span[1] for span, _, _ in pools)
        for x, y in _crossing(self._pools):
            if _meet(x[2], y[2]):
                raise ValueError("pools of the layers, or of K and V, share memory")

    def _call(self, fn: str, stream, *args):
        call = getattr(_abi.kv_lib(), fn)
        if torch.cuda.current_device() == self._index:
            code = call(self._ref, *args, _raw_stream(self._index) if stream is None else stream.cuda_stream)
        else:               # kernels go to the current device
            with torch.cuda.device(self._index):
                code = call(self._ref, *args, _raw_stream(self._index) if stream is None else stream.cuda_stream)
        if code:
            raise _abi.SplitZipError(fn, code)

    def _ints(self, t: torch.Tensor, n: int, what: str, apart: bool = True) -> int:
        """Address of n int32 on the cache's device, apart from what the calls write."""
        if not (t.get_device() == self._index and t.dtype is torch.int32 and t.shape == (n,) and t.is_contiguous()):
            self._check_ints(t, n, what)
        p = t.data_ptr()
        if apart and n:
            end = p + 4 * n
            (s0, e0), (s1, e1), (s2, e2) = self._written
            if p < e0 and s0 < end or p < e1 and s1 < end or p < e2 and s2 < end:
                raise ValueError("the %s share memory with the table, the lengths or the counts" % what)
        return p

    def _check_ints(self, t: torch.Tensor, n: int, what: str) -> None:
        """The same for what the quick look is not content with."""
        if not t.is_cuda or t.device != self.device or t.dtype is not torch.int32 or t.dim() != 1 or t.shape[0] != n or \
                not t.is_contiguous():
            raise ValueError("the %s must be %d contiguous int32 on %s, got %s %s on %s"
                             % (what, n, self.device, t.dtype, tuple(t.shape), t.device))

    def _ready(self) -> None:
        if not self._counted:
            raise ValueError("the pages have not been counted: call count() first")

    def count(self, status: torch.Tensor | None = None, stream=None) -> None:
        """Find out from table and lengths which pages are in use: once before
        the other calls, and again after the table has been written by other
        means.  Entries behind a sequence's length become -1."""
        self._call("splitzip_kv_pages_count", stream, self.caches[0]._status(status))
        self._counted = True

    def fork(self, parents: torch.Tensor, status: torch.Tensor | None = None, stream=None) -> None:
        """Every sequence b becomes a copy of sequence ``parents``[b] (int32
        [batch]), all at once: its pages are named once more, its length is
        taken over.  -1 frees the sequence, b itself leaves it.  Pages that
        several sequences name are read by all; ``resize`` gives each its own
        before one is written."""
        self._ready()
        p = self._ints(parents, self.caches[0].batch, "parents")
        self._call("splitzip_kv_pages_fork", stream, p, self.caches[0]._status(status))

    def resize(self, lens: torch.Tensor, status: torch.Tensor | None = None, stream=None) -> None:
        """The sequences' lengths become ``lens`` (int32 [batch]; it may be the
        cache's own, after an eviction in place).  Pages behind them, or behind
        an old length that is shorter, are freed, then sequences that grow are given pages, the lowest free ones in the
        order of sequences; one that grows within a page that others name is
        given a copy of it (in every layer) first; where all that name it grow,
        the first of them keeps it.  The new tokens are the caller's to append.
        With no page left a sequence gets as long as its pages hold, and stays
        as it was where the page it would write in is still another's
        (KV_NO_PAGE; compare ``lens`` of the cache).

        A length that was made greater in place (``lens += 1``, then
        ``resize(lens)``) grows from the one that the last call here left.
        Between two calls a length may be cut in place or made greater, not cut
        and then made greater: that it grew back over pages that others name
        is not seen.  Layers are evicted from in place one after another, each
        with the lengths of before put back (see ``KVCache.evict``)."""
        self._ready()
        first = self.caches[0]
        own = lens.data_ptr() == first.args.lens and first.batch > 0
        p = self._ints(lens, first.batch, "lengths", not own)
        self._call("splitzip_kv_pages_resize", stream, p, first._status(status))

    def compact(self, moved: torch.Tensor | None = None, used: torch.Tensor | None = None,
                status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Move pages so that those in use are the first ones of the pools (in
        every layer), the table following.  Returns ``used`` (int32 [1]), their
        number; ``moved`` (int32 [pages]) receives every page's new number, -1
        for free ones."""
        self._ready()
        first = self.caches[0]
        m = None if moved is None else self._ints(moved, first.args.num_pages, "new numbers")
        if used is None:
            with torch.cuda.stream(stream):
                used = torch.empty(1, dtype=torch.int32, device=self.device)
        u = self._ints(used, 1, "number of pages")
        if m is not None and m <= u < m + 4 * first.args.num_pages:
            raise ValueError("the number of pages lies in their new numbers")
        self._call("splitzip_kv_pages_compact", stream, m, u, first._status(status))
        return used

    def copy(self, src: torch.Tensor, dst: torch.Tensor, to: "KVPages | None" = None,
             status: torch.Tensor | None = None, stream=None) -> None:
        """Copy K and V of pages ``src`` (int32 [n]) to pages ``dst`` of the
        same pools, or of those of ``to`` (as many layers and pages of the same
        shape, stored in any order), in every layer.  No page is written twice,
        nor one that is read.  Tables, lengths and counts stay as they are."""
        if src.dim() != 1:
            raise ValueError("the pages must be a list, got %s" % (tuple(src.shape),))
        first = self.caches[0]
        if to is None:
            to = self
        elif to is not self:
            if len(to.caches) != len(self.caches) or to._kind != self._kind:
                raise ValueError("the other pages differ in layers, shape, dtype or device")
            self._apart_from(to)
        n = src.shape[0]
        s, d = self._ints(src, n, "pages read", False), self._ints(dst, n, "pages written", False)
        self._call("splitzip_kv_pages_copy", stream, ctypes.byref(to.args), s, d, n, first._status(status))

    def _apart_from(self, to: "KVPages") -> None:
        """Refuses pools that share memory with those of ``to`` without being them."""
        mine, other = self._pools, to._pools
        if self._reach[0] >= to._reach[1] or to._reach[0] >= self._reach[1]:
            return
        both = sorted([(*p, 0) for p in mine] + [(*p, 1) for p in other], key=lambda x: x[0])
        for (_, x, s, a), (_, y, t, b) in _crossing(both):
            if a != b and not (x == y and s.data_ptr() == t.data_ptr() and s.shape == t.shape and s.stride() == t.stride()) and \
                    _meet(s, t):
                raise ValueError("the pages to be written share memory with other ones")


def _crossing(pools):
    """Pairs whose memory ranges cross, of entries that begin with (start, end) and are sorted by it."""
    for i, x in enumerate(pools):
        for y in pools[i + 1:]:
            if y[0][0] >= x[0][1]:
                break
            yield x, y
