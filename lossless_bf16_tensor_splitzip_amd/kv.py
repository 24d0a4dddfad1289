"""Tensor-level calls of the paged key-value cache: marshalling of torch
tensors (device memory and streams only) into the C ABI of
include/splitzip_kv.h.  Copies, attention and eviction run entirely in the HIP
kernels.

    cache = KVCache(k_pages, v_pages, table, lens)
    ws = KVWorkspace(cache, heads)
    lens += 1                              # the step's tokens
    cache.append(k, v, cu)                 # their K and V
    out = cache.attend(q, ws)              # one new token per sequence
    out = cache.attend_shared(q, cu, shared, sws)    # where sequences begin alike

The pools are [pages, kv_heads, page_size, head_dim]; a pool stored
[pages, page_size, kv_heads, head_dim] is passed as its transpose(1, 2).
Nothing here computes gradients: a cache is what a serving step keeps.
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd import forward_ad as _forward

from . import _abi
from .codec import _device_or_pinned, _same_gpu, _status_ptr

_DTYPES = {torch.bfloat16: _abi.KV_BF16, torch.float16: _abi.KV_FP16}
_raw_stream = torch._C._cuda_getCurrentRawStream     # an int, without making a Stream object
_NO_MASS = (None, None, 0, 0, 0, 0, 0)


def _strides(t: torch.Tensor, what: str, multiple: int = 8):
    """Strides of all dimensions but the last, which must be contiguous; those
    of a dimension of one entry are never used and given as 0."""
    size, stride = t.shape, t.stride()
    if stride[-1] != 1 and size[-1] > 1:
        raise ValueError("the last dimension of the %s must be contiguous" % what)
    out = [st if n > 1 else 0 for n, st in zip(size[:-1], stride[:-1])]
    if multiple > 1:
        if t.data_ptr() % (2 * multiple):
            raise ValueError("the %s must be %d-byte aligned" % (what, 2 * multiple))
        for st in out:
            if st % multiple:
                raise ValueError("the strides of the %s must be multiples of %d elements, got %s"
                                 % (what, multiple, tuple(stride)))
    return out


def _place(t: torch.Tensor, what: str, written: bool):
    """Address and strides of a 16-bit tensor of three dimensions, checked as
    ``_strides`` and, where it is written, ``_no_overlap`` do; those two run
    only where the quick look is not content."""
    p, (s0, s1, s2) = t.data_ptr(), t.stride()
    if s2 != 1 or (s0 | s1 | p >> 1) & 7:
        s0, s1 = _strides(t, what)
    if written and not (s1 >= t.shape[2] and s0 >= s1 * t.shape[1]):
        _no_overlap(t, what)
    return p, s0, s1


def _no_overlap(t: torch.Tensor, what: str) -> None:
    """Refuses a written tensor two of whose elements share memory (an
    expanded one)."""
    reach = 0
    for st, n in sorted((st, n) for n, st in zip(t.shape, t.stride()) if n > 1):
        if st <= reach:
            raise ValueError("elements of the %s overlap in memory" % what)
        reach += st * (n - 1)


def _span(t: torch.Tensor):
    first = t.data_ptr()
    return first, first + t.element_size() * (1 + sum((n - 1) * st for n, st in zip(t.shape, t.stride())))


def _reach(size, s0: int, s1: int) -> int:
    """Bytes from the first to behind the last element of a 16-bit tensor of
    three dimensions, the last contiguous (0 entries: no more than one)."""
    return 2 * ((size[0] - 1) * s0 + (size[1] - 1) * s1 + size[2])


def _meet(x: torch.Tensor, y: torch.Tensor) -> bool:
    """Whether some element of one tensor shares memory with one of the other
    (interleaved ones need not).  Their distance is a sum of strides, each
    taken c times; of the largest stride only the c that the others can bring
    back to 0 are looked at, and so on down."""
    (p, p_end), (q, q_end) = _span(x), _span(y)
    if not x.numel() or not y.numel() or p_end <= q or q_end <= p:
        return False
    ex, ey = x.element_size(), y.element_size()
    steps = {}
    for t, side in ((x, 1), (y, 0)):
        for n, st in zip(t.shape, t.stride()):
            if n > 1 and st:
                steps.setdefault(st * t.element_size(), [0, 0])[side] += n - 1
    steps = sorted(steps.items(), reverse=True)
    below = [(0, 0)]
    for st, (less, more) in reversed(steps):
        below.append((below[-1][0] - st * less, below[-1][1] + st * more))
    below.reverse()
    looks = 0

    def found(d, i):
        nonlocal looks
        looks += 1
        if i == len(steps) or looks > 100000:       # strides of no order: taken as meeting
            return i < len(steps) or -ex < d < ey
        st, (less, more) = steps[i]
        low, high = below[i + 1]
        first, last = max(-less, -((d + high + ex - 1) // st)), min(more, (ey - 1 - low - d) // st)
        return any(found(d + st * c, i + 1) for c in range(first, last + 1))

    return found(p - q, 0)


def _same(x: torch.Tensor, y: torch.Tensor) -> bool:
    """Whether two tensors of one shape and type are the same elements."""
    return x.data_ptr() == y.data_ptr() and all(
        a == b for n, a, b in zip(x.shape, x.stride(), y.stride()) if n > 1)


def _plain(t: torch.Tensor, dtype, dims: int, what: str) -> None:
    if not t.is_cuda:
        raise ValueError("the %s must be on the GPU" % what)
    if t.dtype is not dtype:
        raise ValueError("the %s must be %s, got %s" % (what, dtype, t.dtype))
    if t.dim() != dims:
        raise ValueError("the %s must have %d dimensions, got %d" % (what, dims, t.dim()))


def _no_grad(t: torch.Tensor, what: str) -> None:
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError("the %s requires a gradient, and the cache computes none" % what)
    if _forward._current_level >= 0 and _forward.unpack_dual(t).tangent is not None:
        raise ValueError("the %s has a tangent, and the cache computes none" % what)


def _fixed(name: str):
    def get(self):
        return self._tensors[name]

    def put(self, value):
        if value is not self._tensors[name]:
            raise ValueError("the cache's %s stays the tensor it was made with: copy into it" % name)

    return property(get, put)


class KVCache:
    """A paged cache: K and V pools [pages, kv_heads, page_size, head_dim]
    (bfloat16 or float16, last dimension contiguous, other strides multiples
    of 8), ``table`` int32 [batch, max_pages] (rows of their own, not one
    expanded) and ``lens`` int32 [batch].  It holds the caller's tensors and
    allocates nothing; table and lens may be changed between calls.

    Every call takes ``stream`` (None: the current one), on which its tensors
    must be ready and be kept until it has run, and ``status``, an int32 tensor
    that the caller has set to 0: bits _abi.KV_BAD_PAGE (a page number outside
    the pools: its tokens are left out), KV_BAD_LEN (a length outside the table
    or the mass: cut) and KV_BAD_ROWS (rows without a place: left out) are ORed
    into it."""

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor, table: torch.Tensor, lens: torch.Tensor):
        if k_pages.dtype not in _DTYPES:
            raise ValueError("the pools must be bfloat16 or float16, got %s" % k_pages.dtype)
        _plain(k_pages, k_pages.dtype, 4, "K pool")
        _plain(v_pages, k_pages.dtype, 4, "V pool")
        _plain(table, torch.int32, 2, "page table")
        _plain(lens, torch.int32, 1, "lengths")
        if k_pages.shape != v_pages.shape:
            raise ValueError("the pools differ in shape: %s and %s" % (tuple(k_pages.shape), tuple(v_pages.shape)))
        if table.shape[0] != lens.shape[0] or not lens.is_contiguous():
            raise ValueError("one contiguous length per row of the page table")
        pages, kv_heads, page_size, dim = k_pages.shape
        if pages < 1 or kv_heads < 1 or page_size < 1:
            raise ValueError("the pools are empty: %s" % (tuple(k_pages.shape),))
        if dim % 8 or not 8 <= dim <= 256:
            raise ValueError("head_dim must be a multiple of 8 in 8..256, got %d" % dim)
        if table.shape[1] * page_size >= 1 << 31:
            raise ValueError("a sequence's table reaches 2^31 tokens")
        row = _strides(table, "page table", 1)[0]
        if table.shape[0] > 1 and row < table.shape[1]:
            raise ValueError("rows of the page table overlap in memory: %d pages, %d apart" % (table.shape[1], row))
        for t, what in ((k_pages, "K pool"), (v_pages, "V pool")):
            _no_overlap(t, what)
            _no_grad(t, what)
        _same_gpu(k_pages.device, v_pages, table, lens)
        self._tensors = {"k_pages": k_pages, "v_pages": v_pages, "table": table, "lens": lens}
        self.device, self.dtype = k_pages.device, k_pages.dtype
        self.batch, self.max_pages = table.shape
        self.kv_heads, self.page_size, self.head_dim = kv_heads, page_size, dim
        ks, vs = _strides(k_pages, "K pool"), _strides(v_pages, "V pool")
        self.args = _abi.KVCacheArgs(k_pages.data_ptr(), v_pages.data_ptr(), *ks, *vs, table.data_ptr(),
                                     row, lens.data_ptr(), pages, page_size, kv_heads, dim, self.batch,
                                     self.max_pages, _DTYPES[self.dtype], 0)
        self._ref = ctypes.byref(self.args)
        self._index = self.device.index
        self._row, self._cu, self._heads = (kv_heads, dim), (self.batch + 1,), (self.batch, kv_heads)
        self._spans = _span(k_pages), _span(v_pages), _span(lens)
        # pools that share memory (a latent that is K and V) are read like others;
        # one pool as both can be written where K and V get the same values
        self._one_pool = (k_pages.data_ptr(), ks) == (v_pages.data_ptr(), vs)
        self._pools_meet = self._one_pool or _meet(k_pages, v_pages)
        self._shape = (self.batch, kv_heads, dim, self.dtype, self.device)

    # The kernels are given these tensors' memory once: in-place changes reach
    # them (cache.lens += 1, cache.table.copy_(...)), other tensors do not.
    k_pages, v_pages, table, lens = (_fixed(name) for name in ("k_pages", "v_pages", "table", "lens"))

    def _call(self, fn: str, stream, *args):
        call = getattr(_abi.kv_lib(), fn)
        if torch.cuda.current_device() == self._index:
            code = call(self._ref, *args, _raw_stream(self._index) if stream is None else stream.cuda_stream)
        else:               # kernels go to the current device
            with torch.cuda.device(self._index):
                code = call(self._ref, *args, _raw_stream(self._index) if stream is None else stream.cuda_stream)
        if code:
            raise _abi.SplitZipError(fn, code)

    def _here(self, t: torch.Tensor, what: str) -> None:
        if t.device != self.device:
            raise ValueError("the %s must be on %s, got %s" % (what, self.device, t.device))

    def _rows(self, k, v, cu, start, written: bool):
        size = k.shape
        if not (k.dtype is v.dtype is self.dtype and size == v.shape and len(size) == 3 and size[1:] == self._row and
                k.device == v.device == cu.device == self.device and cu.dtype is torch.int32 and cu.shape == self._cu and
                start is None and cu.is_contiguous() and not (k.requires_grad or v.requires_grad) and
                _forward._current_level < 0):
            self._check_rows(k, v, cu, start)
        kp, k0, k1 = _place(k, "K rows", written)
        vp, v0, v1 = _place(v, "V rows", written)
        if written and vp < kp + _reach(size, k0, k1) and kp < vp + _reach(size, v0, v1) and _meet(k, v):
            raise ValueError("the K rows and the V rows overlap in memory")
        if self._pools_meet and not written and not (self._one_pool and _same(k, v)):
            raise ValueError("K and V rows that differ cannot be written to pools that share memory")
        return ctypes.byref(_abi.KVRows(kp, vp, k0, k1, v0, v1, size[0], 0, cu.data_ptr(),
                                        None if start is None else start.data_ptr()))

    def _check_rows(self, k, v, cu, start):
        """The same one by one, for what the quick look is not content with."""
        for t, what in ((k, "K rows"), (v, "V rows")):
            if t.is_cuda:
                self._here(t, what)
            else:
                _device_or_pinned(t, what)
            if t.dtype is not self.dtype or t.dim() != 3 or tuple(t.shape[1:]) != self._row:
                raise ValueError("the %s must be %s [rows, %d, %d], got %s %s"
                                 % ((what, self.dtype) + self._row + (t.dtype, tuple(t.shape))))
            _no_grad(t, what)
        if k.shape[0] != v.shape[0]:
            raise ValueError("K and V must have the same number of rows")
        for t, n, what in ((cu, self.batch + 1, "row ranges"), (start, self.batch, "first positions")):
            if t is None and what == "first positions":
                continue
            _plain(t, torch.int32, 1, what)
            self._here(t, what)
            if t.shape[0] != n or not t.is_contiguous():
                raise ValueError("the %s need %d contiguous entries" % (what, n))

    def append(self, k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor, start: torch.Tensor | None = None,
               status: torch.Tensor | None = None, stream=None) -> None:
        """Write rows ``k`` and ``v`` [rows, kv_heads, head_dim] (device or
        pinned host memory) into the cache.  Rows cu[b] .. cu[b+1]-1 (``cu``
        int32 [batch + 1]) go to positions start[b], start[b]+1, ... of
        sequence b, whatever its length; with ``start`` None they are its last
        ones: ``lens`` counts them already.  Rows behind cu[batch] are not read."""
        rows = self._rows(k, v, cu, start, False)
        self._call("splitzip_kv_append", stream, rows, self._status(status))

    def gather(self, k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor, start: torch.Tensor | None = None,
               status: torch.Tensor | None = None, stream=None) -> None:
        """Copy cached tokens into rows ``k`` and ``v``, placed as in
        ``append``.  Rows behind cu[batch] are left as they are."""
        rows = self._rows(k, v, cu, start, True)
        self._call("splitzip_kv_gather", stream, rows, self._status(status))

    def _status(self, status):
        if status is None:
            return None
        _same_gpu(self.device, status)
        return _status_ptr(status)

    def _mass(self, mass, what: str, written: bool):
        _plain(mass, torch.float32, 3, what)
        self._here(mass, what)
        if mass.shape[0] != self.batch or mass.shape[1] != self.kv_heads:
            raise ValueError("the %s must be [%d, %d, tokens], got %s"
                             % (what, self.batch, self.kv_heads, tuple(mass.shape)))
        _no_grad(mass, what)
        if written:
            _no_overlap(mass, what)
        return _strides(mass, what, 1)

    def _mass_pair(self, mass, mass_out):
        """Addresses, strides and entries of a mass that is read (or None) and
        one that is written (the same one, or one apart from it)."""
        if mass_out is None:
            mass_out = mass
        size, f32 = mass_out.shape, torch.float32
        if (len(size) == 3 and size[:2] == self._heads and mass_out.dtype is f32 and mass_out.device == self.device and
                _forward._current_level < 0):
            p, (s0, s1, s2) = mass_out.data_ptr(), mass_out.stride()
            if s2 == 1 and s1 >= size[2] and s0 >= s1 * size[1] and not mass_out.requires_grad:
                if mass is mass_out:
                    return p, p, s0, s1, s0, s1, size[2]
                if mass is None:
                    return None, p, 0, 0, s0, s1, size[2]
                if (mass.shape == size and mass.dtype is f32 and mass.device == self.device and not mass.requires_grad and
                        mass.stride() == (s0, s1, 1)):
                    q, reach = mass.data_ptr(), 4 * s0 * size[0]
                    if q + reach <= p or p + reach <= q:
                        return q, p, s0, s1, s0, s1, size[2]
        return self._check_masses(mass, mass_out)

    def _check_masses(self, mass, mass_out):
        """The same one by one, for what the quick look is not content with."""
        out_strides = self._mass(mass_out, "mass output", True)
        if mass is None:
            return (None, mass_out.data_ptr(), 0, 0, *out_strides, mass_out.shape[2])
        strides = out_strides if mass is mass_out else self._mass(mass, "mass", False)
        if mass.shape[2] != mass_out.shape[2]:
            raise ValueError("the masses differ in length: %d and %d" % (mass.shape[2], mass_out.shape[2]))
        if (mass.data_ptr(), strides) != (mass_out.data_ptr(), out_strides) and _meet(mass, mass_out):
            raise ValueError("the mass and its output overlap without being the same")
        return (mass.data_ptr(), mass_out.data_ptr(), *strides, *out_strides, mass.shape[2])

    def attend(self, q: torch.Tensor, ws: "KVWorkspace", out: torch.Tensor | None = None, scale: float | None = None,
               window: int | None = None, sinks: int = 0, lse: torch.Tensor | None = None,
               mass: torch.Tensor | None = None, mass_out: torch.Tensor | None = None,
               status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Attention of one new token per sequence, ``q`` [batch, heads,
        head_dim], over its cached tokens: all, or with ``window`` the last
        ``window`` and the first ``sinks``.  ``scale`` defaults to
        head_dim ** -0.5.  Returns ``out``, shaped like q; a sequence with
        nothing visible gives zeros; ``out`` may be ``q``, else they must not
        overlap.

        ``lse`` (float32 [batch, heads]) receives the log of the sum of
        exponentials.  With ``mass`` (float32 [batch, kv_heads, tokens]) the
        weight every token received, summed over its KV head's query heads, is
        added to it: in place, or into ``mass_out``, whose entries up to the
        length are all written (with ``mass_out`` alone, starting from 0)."""
        size, index = q.shape, self._index
        if q.dtype is not self.dtype or len(size) != 3 or size[0] != self.batch or size[2] != self.head_dim:
            raise ValueError("the queries must be %s [%d, heads, %d], got %s %s"
                             % (self.dtype, self.batch, self.head_dim, q.dtype, tuple(size)))
        if not q.get_device() == ws.buf.get_device() == index:
            self._here(q, "queries")
            self._here(ws.buf, "workspace")
        if q.requires_grad or _forward._current_level >= 0:
            _no_grad(q, "queries")
        heads = size[1]
        if heads < 1 or heads % self.kv_heads:
            raise ValueError("%d query heads do not divide over %d KV heads" % (heads, self.kv_heads))
        if window is None:
            window = _abi.KV_ALL
        elif not 0 <= window < 1 << 31:
            raise ValueError("the window must be in 0..2^31-1, got %d" % window)
        if not 0 <= sinks < 1 << 31:
            raise ValueError("the sinks must be in 0..2^31-1, got %d" % sinks)
        if out is not None:
            if out.dtype is not self.dtype or out.shape != size:
                raise ValueError("the output must be shaped like the queries")
            if out.get_device() != index:
                self._here(out, "output")
            if out.requires_grad or _forward._current_level >= 0:
                _no_grad(out, "output")
        if lse is not None:
            _plain(lse, torch.float32, 2, "lse")
            if tuple(lse.shape) != (self.batch, heads) or not lse.is_contiguous():
                raise ValueError("lse must be contiguous [%d, %d]" % (self.batch, heads))
            self._here(lse, "lse")
            _no_grad(lse, "lse")
        masses = _NO_MASS if mass is None and mass_out is None else self._mass_pair(mass, mass_out)
        if masses[1] == 0:      # a mass of no tokens has no address: one that is not written to stands for it
            masses = (None, self.args.lens, 0, 0, 0, 0, 0)
        qp, q0, q1 = _place(q, "queries", False)
        if out is None:
            with torch.cuda.stream(stream):
                out = torch.empty(size, dtype=q.dtype, device=self.device)
        op, o0, o1 = _place(out, "output", True)
        # the queries themselves, or apart from them: another workgroup's output
        # must not land in queries that are still to be read
        if (out is not q and op < qp + 2 * ((size[0] - 1) * q0 + (heads - 1) * q1 + size[2]) and
                qp < op + _reach(size, o0, o1) and not _same(q, out) and _meet(q, out)):
            raise ValueError("the output overlaps the queries without being the same")
        query = _abi.KVQuery(qp, q0, q1, op, o0, o1, None if lse is None else lse.data_ptr(), *masses[:6], heads, window,
                             sinks, self.head_dim ** -0.5 if scale is None else scale, masses[6], 0)
        self._call("splitzip_kv_attend", stream, ctypes.byref(query), ws.buf.data_ptr(), ws.nbytes, self._status(status))
        return out

    def attend_shared(self, q: torch.Tensor, cu: torch.Tensor, shared: torch.Tensor, ws: "KVSharedWorkspace",
                      out: torch.Tensor | None = None, scale: float | None = None, lse: torch.Tensor | None = None,
                      status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """``attend`` over all cached tokens for a batch whose sequences begin
        alike: sequences cu[g] .. cu[g+1]-1 (``cu`` int32 [groups + 1],
        ascending) have their first ``shared``[g] tokens (int32 [groups], no
        more than the first of them has) in common, and these are read through
        the table row of the group's first sequence, once for up to 128 query
        rows of a KV head where they are many (their weights are rounded to the
        cache's type then), for 16 or 32 where they are few, by each sequence
        where those have no room for two.  The others need the same values
        there, as after ``KVPages.fork``; one that is shorter attends on its
        own, as do sequences outside ``cu``, and all of a group whose first
        sequence has ended: begin it with one that goes on.  Which form is
        taken goes by the shapes, the groups and the table's width, not by the
        lengths: a table much wider than its sequences gets the form for long
        ones.  ``out`` and ``lse`` as in ``attend``."""
        size, index = q.shape, self._index
        if q.dtype is not self.dtype or len(size) != 3 or size[0] != self.batch or size[2] != self.head_dim:
            raise ValueError("the queries must be %s [%d, heads, %d], got %s %s"
                             % (self.dtype, self.batch, self.head_dim, q.dtype, tuple(size)))
        if not q.get_device() == ws.buf.get_device() == cu.get_device() == shared.get_device() == index:
            for t, what in ((q, "queries"), (ws.buf, "workspace"), (cu, "group ranges"), (shared, "tokens in common")):
                self._here(t, what)
        if q.requires_grad or _forward._current_level >= 0:
            _no_grad(q, "queries")
        heads = size[1]
        if heads < 1 or heads % self.kv_heads:
            raise ValueError("%d query heads do not divide over %d KV heads" % (heads, self.kv_heads))
        groups = shared.shape[0] if shared.dim() == 1 else -1
        if not (cu.dtype is shared.dtype is torch.int32 and cu.shape == (groups + 1,) and cu.is_contiguous() and
                shared.is_contiguous()):
            raise ValueError("group ranges and tokens in common must be contiguous int32 [groups + 1] and [groups], got %s %s and %s %s"
                             % (cu.dtype, tuple(cu.shape), shared.dtype, tuple(shared.shape)))
        if groups > _abi.KV_MAX_GROUPS:
            raise ValueError("at most %d groups, got %d" % (_abi.KV_MAX_GROUPS, groups))
        if out is not None:
            if out.dtype is not self.dtype or out.shape != size:
                raise ValueError("the output must be shaped like the queries")
            if out.get_device() != index:
                self._here(out, "output")
            if out.requires_grad or _forward._current_level >= 0:
                _no_grad(out, "output")
        if lse is not None and not (lse.dtype is torch.float32 and lse.shape == (self.batch, heads) and
                                    lse.get_device() == index and lse.is_contiguous() and not lse.requires_grad and
                                    _forward._current_level < 0):
            _plain(lse, torch.float32, 2, "lse")
            if tuple(lse.shape) != (self.batch, heads) or not lse.is_contiguous():
                raise ValueError("lse must be contiguous [%d, %d]" % (self.batch, heads))
            self._here(lse, "lse")
            _no_grad(lse, "lse")
        qp, q0, q1 = _place(q, "queries", False)
        if out is None:
            with torch.cuda.stream(stream):
                out = torch.empty(size, dtype=q.dtype, device=self.device)
        op, o0, o1 = _place(out, "output", True)
        if (out is not q and op < qp + 2 * ((size[0] - 1) * q0 + (heads - 1) * q1 + size[2]) and
                qp < op + _reach(size, o0, o1) and not _same(q, out) and _meet(q, out)):
            raise ValueError("the output overlaps the queries without being the same")
        query = _abi.KVQuery(qp, q0, q1, op, o0, o1, None if lse is None else lse.data_ptr(), *_NO_MASS[:6], heads,
                             _abi.KV_ALL, 0, self.head_dim ** -0.5 if scale is None else scale, 0, 0)
        of = _abi.KVGroups(cu.data_ptr(), shared.data_ptr(), groups, 0)
        self._call("splitzip_kv_attend_shared", stream, ctypes.byref(query), ctypes.byref(of), ws.buf.data_ptr(), ws.nbytes,
                   self._status(status))
        return out

    def evict(self, mass: torch.Tensor, budget: int, sinks: int = 0, recent: int = 0, to: "KVCache | None" = None,
              kept: torch.Tensor | None = None, mass_out: torch.Tensor | None = None,
              status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Keep ``budget`` tokens per KV head of every sequence longer than
        that: the first ``sinks``, the last ``recent`` and those of the
        largest ``mass`` between them (equal masses: the earlier token), in
        their order.  In place, or into the pages and lengths of ``to``, which
        share no memory with this cache; ``lens`` (of ``to``) becomes
        min(length, budget), and the mass moves along (in place, or into
        ``mass_out``), 0 behind it.  Returns ``kept``, int32 [batch, kv_heads,
        budget]: the old position of each kept token, -1 behind them.

        Caches of several layers with one ``lens`` (``KVPages``): the first
        eviction in place sets it, so put the lengths back before each further
        layer (``lens.copy_(before)``), or that one finds nothing to evict; then
        ``KVPages.resize(lens)`` frees the pages behind them.  In place, pages
        are written: none that several sequences name (after a fork)."""
        if budget < 1 or budget >= 1 << 31 or sinks < 0 or recent < 0 or sinks + recent > budget:
            raise ValueError("the budget %d must be positive and hold %d sinks and %d recent tokens"
                             % (budget, sinks, recent))
        if to is None:
            to = self
        elif to._shape != self._shape:
            raise ValueError("the destination cache differs in batch, heads, dtype or device")
        if to.max_pages * to.page_size < min(budget, self.max_pages * self.page_size):
            raise ValueError("the destination's table cannot hold %d tokens" % budget)
        if to is not self:
            self._apart(to)
        if to._pools_meet and not (to._one_pool and self._one_pool and to.args.k != self.args.k):
            raise ValueError("the K and V pools of the destination share memory")
        shape = (self.batch, self.kv_heads, budget)
        if mass is None:
            raise ValueError("an eviction needs the mass")
        if kept is not None and not (kept.shape == shape and kept.dtype is torch.int32 and kept.device == self.device and
                                     kept.is_contiguous()):
            _plain(kept, torch.int32, 3, "kept positions")
            if tuple(kept.shape) != shape or not kept.is_contiguous():
                raise ValueError("the kept positions must be contiguous %s" % (shape,))
            self._here(kept, "kept positions")
        masses = self._mass_pair(mass, mass_out)
        if kept is None:
            with torch.cuda.stream(stream):
                kept = torch.empty(shape, dtype=torch.int32, device=self.device)
        args = _abi.KVBudget(*masses[:6], kept.data_ptr(), budget, sinks, recent, masses[6])
        self._call("splitzip_kv_evict", stream, to._ref, ctypes.byref(args), self._status(status))
        return kept


    def _apart(self, to: "KVCache") -> None:
        """Refuses a destination that would overwrite what is still to be read
        (one with a start in common is the library's to judge: the cache itself
        in all fields, or refused)."""
        a, b = self.args, to.args
        if a.k == b.k or a.v == b.v or a.table == b.table or a.lens == b.lens:
            return
        (k, k_end), (v, v_end), (n, n_end) = self._spans
        (tk, tk_end), (tv, tv_end), (tn, tn_end) = to._spans
        if (k < tk_end and tk < k_end or k < tv_end and tv < k_end or v < tk_end and tk < v_end or
                v < tv_end and tv < v_end or n < tn_end and tn < n_end):
            for x, y in (("k_pages", "k_pages"), ("k_pages", "v_pages"), ("v_pages", "k_pages"),
                         ("v_pages", "v_pages"), ("lens", "lens")):
                if _meet(self._tensors[x], to._tensors[y]):
                    raise ValueError("the destination shares memory with the cache (%s and %s)" % (y, x))


class KVWorkspace:
    """Device scratch for ``KVCache.attend`` on caches shaped like ``cache``
    with ``heads`` query heads (``mass``: also for calls that ask for the
    mass).  One workspace per stream that runs such calls concurrently."""

    def __init__(self, cache: KVCache, heads: int, mass: bool = False):
        mass_len = cache.max_pages * cache.page_size if mass else 0
        self.nbytes = _abi.splitzip_kv_attend_workspace_size(cache.args, heads, mass_len)
        if not self.nbytes:
            raise ValueError("%d query heads do not divide over %d KV heads" % (heads, cache.kv_heads))
        self.buf = self._buffer(self.nbytes, cache.device)

    def _buffer(self, nbytes: int, device) -> torch.Tensor:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


class KVSharedWorkspace(KVWorkspace):
    """Device scratch for ``KVCache.attend_shared`` on caches shaped like
    ``cache`` with ``heads`` query heads and up to ``groups`` groups.  One
    workspace per stream that runs such calls concurrently."""

    def __init__(self, cache: KVCache, heads: int, groups: int = _abi.KV_MAX_GROUPS):
        self.nbytes = _abi.splitzip_kv_shared_workspace_size(cache.args, heads, groups)
        if not self.nbytes:
            raise ValueError("no workspace for %d query heads over %d KV heads in %d groups" % (heads, cache.kv_heads, groups))
        self.buf = self._buffer(self.nbytes, cache.device)
