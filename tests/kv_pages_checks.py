"""What the page operators and the attention over sequences that begin alike
refuse.  Written like kv_checks, for a run without a GPU and one with it."""
import torch
from torch.autograd import forward_ad

import lossless_bf16_tensor_splitzip_amd as S
import kv_reference as R
from kv_checks import refused


def layers(new, to_gpu, runs):
    """Caches that are not layers of one model."""
    m = to_gpu(R.make([20, 3], 2, 64, 16, torch.bfloat16, seed=1))
    far = to_gpu(R.make([20, 3], 2, 64, 16, torch.bfloat16, seed=2))
    k, v, t, n = m.gk, m.gv, m.gtable, m.glens
    refused(S.KVPages, [])
    refused(S.KVPages, [m.cache] * 1025)
    refused(S.KVPages, [m.cache, far.cache])                                     # tables of their own
    refused(S.KVPages, [m.cache, S.KVCache(far.gk, far.gv, t, far.glens)])       # lengths
    refused(S.KVPages, [m.cache, S.KVCache(far.gk[:-1], far.gv[:-1], t, n)])     # fewer pages
    refused(S.KVPages, [m.cache, S.KVCache(far.gk.transpose(1, 2).contiguous().transpose(1, 2), far.gv, t, n)])
    refused(S.KVPages, [m.cache, m.cache])                                       # one layer's pools
    refused(S.KVPages, [m.cache, S.KVCache(far.gk, v, t, n)])
    refused(S.KVPages, S.KVCache(k, k, t, n))                                    # one pool as K and V
    refused(S.KVPages, S.KVCache(k[:-1], k[1:], t, n))
    both = new(torch.zeros, 6, 4, 2, 16, 64, dtype=torch.bfloat16)               # layers that interleave
    pages = S.KVPages([S.KVCache(both[:, 0], both[:, 1], t, n), S.KVCache(both[:, 2], both[:, 3], t, n)])
    runs(pages.count)
    assert pages.refs.dtype is torch.int32 and pages.refs.shape == (6,)


def lists(new, to_gpu, runs):
    """Parents, lengths and page numbers."""
    m = to_gpu(R.make([20, 3], 2, 64, 16, torch.bfloat16, seed=1))
    pages = S.KVPages(m.cache)
    good = new(torch.tensor, [0, 0], dtype=torch.int32)
    used = new(torch.zeros, 1, dtype=torch.int32)
    moved = new(torch.zeros, m.gk.shape[0], dtype=torch.int32)
    for call in (lambda: pages.fork(good), lambda: pages.resize(good), lambda: pages.compact(used=used)):
        refused(call)                                                            # not counted yet
    pages._counted = True
    refused(pages.count, status=new(torch.zeros, 1))
    for fn in (pages.fork, pages.resize):
        refused(fn, good[:1])
        refused(fn, good.long())
        refused(fn, good.cpu())
        refused(fn, new(torch.zeros, 4, dtype=torch.int32)[::2])
        refused(fn, new(torch.zeros, 2, 1, dtype=torch.int32))
        refused(fn, m.gtable.reshape(-1)[:2])                                    # written while it is read
        refused(fn, pages.refs[:2])
        refused(fn, good, status=good.float())
        runs(fn, good)
    refused(pages.fork, m.glens)
    runs(pages.resize, m.glens)                                                  # its own lengths
    refused(pages.compact, used=new(torch.zeros, 2, dtype=torch.int32))
    refused(pages.compact, moved=moved[1:], used=used)
    refused(pages.compact, moved=moved, used=moved[:1])
    refused(pages.compact, moved=pages.refs, used=used)
    refused(pages.compact, used=m.glens[:1])
    runs(pages.compact, moved=moved, used=used)
    a, b = new(torch.tensor, [0, 1], dtype=torch.int32), new(torch.tensor, [2, 3], dtype=torch.int32)
    refused(pages.copy, a, b[:1])
    refused(pages.copy, a.long(), b)
    refused(pages.copy, a, b.cpu())
    refused(pages.copy, a.reshape(1, 2), b.reshape(1, 2))
    runs(pages.copy, a, b)
    far = to_gpu(R.make([20, 3], 2, 64, 16, torch.bfloat16, layout="nhd", seed=2))
    runs(pages.copy, a, b, to=S.KVPages(far.cache))
    for other in (R.make([20], 2, 64, 8, torch.bfloat16), R.make([20], 1, 64, 16, torch.bfloat16),
                  R.make([20], 2, 72, 16, torch.bfloat16), R.make([20], 2, 64, 16, torch.float16)):
        refused(pages.copy, a, b, to=S.KVPages(to_gpu(other).cache))
    refused(pages.copy, a, b, to=S.KVPages(S.KVCache(m.gk[1:], far.gv[:-1], m.gtable, m.glens)))
    same = S.KVPages(S.KVCache(m.gk, m.gv, far.gtable, far.glens))               # the same pools
    runs(pages.copy, a, b, to=same)


def groups(new, to_gpu, runs):
    """Attention over sequences that begin alike."""
    m = to_gpu(R.make([20, 3], 2, 64, 16, torch.bfloat16, heads=4, seed=1))
    q, ws = m.gq, S.KVSharedWorkspace(m.cache, 4, 1)
    cu, shared = new(torch.tensor, [0, 2], dtype=torch.int32), new(torch.tensor, [3], dtype=torch.int32)
    out = torch.zeros_like(q)
    for heads, n in ((3, 1), (0, 1), (4, 65536), (65536 * 2, 1)):
        refused(S.KVSharedWorkspace, m.cache, heads, n)

    def no(*args, **kw):
        refused(m.cache.attend_shared, *args, out=kw.pop("out", out), **kw)

    no(q.float(), cu, shared, ws)
    no(q[:1], cu, shared, ws)
    no(q[:, :3], cu, shared, ws)
    no(q.cpu(), cu, shared, ws)
    no(q, cu.long(), shared, ws)
    no(q, cu, shared.long(), ws)
    no(q, cu[:1], shared, ws)
    no(q, cu, cu, ws)
    no(q, cu.cpu(), shared, ws)
    no(q, cu, shared.cpu(), ws)
    no(q, cu, shared.reshape(1, 1), ws)
    no(q, new(torch.zeros, 4, dtype=torch.int32)[::2], shared, ws)
    no(q, new(torch.zeros, 65537, dtype=torch.int32), new(torch.zeros, 65536, dtype=torch.int32), ws)
    no(q, cu, shared, ws, out=out[:, :2])
    no(q, cu, shared, ws, out=out.float())
    no(q, cu, shared, ws, out=torch.zeros_like(q[:, :1]).expand(-1, 4, -1))
    no(q, cu, shared, ws, lse=new(torch.zeros, 2, 3))
    no(q, cu, shared, ws, scale=float("inf"))
    no(q, cu, shared, ws, status=new(torch.zeros, 1))
    no(q.clone().requires_grad_(), cu, shared, ws)
    packed = new(torch.zeros, 3, 8, 64, dtype=torch.bfloat16)
    no(packed[:2, :4], cu, shared, ws, out=packed[1:, :4])
    small = S.KVSharedWorkspace(m.cache, 4, 1)
    small.nbytes = 64
    no(q, cu, shared, small)
    with forward_ad.dual_level():
        no(forward_ad.make_dual(q.clone(), torch.ones_like(q)), cu, shared, ws)
    runs(m.cache.attend_shared, packed[:2, :4], cu, shared, ws, out=packed[:2, 4:])
    runs(m.cache.attend_shared, q, cu, shared, ws, out=out)
    runs(m.cache.attend_shared, q, cu[:1], shared[:0], ws, out=out)


PARTS = ("layers", "lists", "groups")
