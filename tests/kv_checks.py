"""What the tensor-level calls of the key-value cache refuse, for a run without
a GPU and one with it: ``new(make, ...)`` makes a tensor there, ``to_gpu`` a
cache, and ``runs`` a call that is accepted."""
import pytest
import torch

import lossless_bf16_tensor_splitzip_amd as S
from lossless_bf16_tensor_splitzip_amd import _abi
import kv_reference as R


def refused(fn, *args, **kw):
    """Argument errors of the binding or of the library: never a launch."""
    with pytest.raises((ValueError, S.SplitZipError)) as e:
        fn(*args, **kw)
    assert not isinstance(e.value, S.SplitZipError) or e.value.status in (_abi.ERR_INVALID, _abi.ERR_WORKSPACE)


def caches(new, to_gpu, runs):
    m = to_gpu(R.make([20, 3], 2, 64, 16, torch.bfloat16, heads=4, seed=1))
    k, v, t, n = m.gk, m.gv, m.gtable, m.glens
    refused(S.KVCache, k.float(), v.float(), t, n)
    refused(S.KVCache, k, v.to(torch.float16), t, n)
    refused(S.KVCache, k[:-1], v, t, n)
    refused(S.KVCache, k[0], v[0], t, n)
    refused(S.KVCache, k, v, t.long(), n)
    refused(S.KVCache, k, v, t, n.long())
    refused(S.KVCache, k, v, t, n[:1])
    refused(S.KVCache, k, v, t.t(), new(torch.zeros, t.shape[1], dtype=torch.int32))
    refused(S.KVCache, k.cpu(), v.cpu(), t, n)
    refused(S.KVCache, k, v, t.cpu(), n)
    refused(S.KVCache, k.transpose(2, 3), v.transpose(2, 3), t, n)
    refused(S.KVCache, k[..., 4:60], v[..., 4:60], t, n)                  # not 16-byte aligned
    refused(S.KVCache, k[..., :60], v[..., :60], t, n)                    # 60 is no multiple of 8
    refused(S.KVCache, k[:1].expand(4, -1, -1, -1), v[:4], t, n)          # pages that are one page
    odd = new(torch.zeros, 6, 2, 16, 68, dtype=torch.bfloat16)[..., :64]
    refused(S.KVCache, odd, odd.clone(), t, n)                            # rows 136 bytes apart
    wide = new(torch.zeros, 2, 1, 16, 264, dtype=torch.bfloat16)
    refused(S.KVCache, wide, wide.clone(), t, n)
    refused(S.KVCache, k.requires_grad_(), v, t, n)
    k.requires_grad_(False)


    m = to_gpu(R.make([20, 3], 2, 64, 16, torch.bfloat16, seed=1))
    m.cache.lens += 1                                                     # in place: the same tensor
    assert m.cache.lens is m.glens and m.glens.tolist() == [21, 4]
    for name in ("lens", "table", "k_pages", "v_pages"):
        refused(setattr, m.cache, name, getattr(m.cache, name).clone())


def rows(new, to_gpu, runs):
    m = to_gpu(R.make([20, 3], 2, 64, 16, torch.bfloat16, heads=4, seed=1))
    k = new(torch.zeros, 4, 2, 64, dtype=torch.bfloat16)
    cu = new(torch.tensor, [0, 2, 4], dtype=torch.int32)
    for fn in (m.cache.append, m.cache.gather):
        refused(fn, k, k[:3], cu)
        refused(fn, k.to(torch.float16), k, cu)
        refused(fn, k, k.view(4, 1, 128), cu)
        refused(fn, k, k.clone(), cu[:2])
        refused(fn, k, k.clone(), cu.long())
        refused(fn, k, k.clone(), cu.cpu())
        refused(fn, k, k.clone(), new(torch.zeros, 6, dtype=torch.int32)[::2])
        refused(fn, k, k.clone(), cu, start=cu)
        refused(fn, k.cpu(), k.cpu(), cu)                                 # pageable host memory
        refused(fn, k, k.clone(), cu, status=new(torch.zeros, 1))
    refused(m.cache.gather, k[:1].expand(4, -1, -1), k.clone(), cu)       # rows written over each other
    runs(m.cache.append, k[:1].expand(4, -1, -1), k, cu)                  # read, one row for all is fine


def queries(new, to_gpu, runs):
    m = to_gpu(R.make([20, 3], 2, 64, 16, torch.bfloat16, heads=4, seed=1))
    ws = S.KVWorkspace(m.cache, 4)
    q = m.gq
    refused(S.KVWorkspace, m.cache, 3)
    refused(S.KVWorkspace, m.cache, 0)
    refused(m.cache.attend, q.float(), ws)
    refused(m.cache.attend, q[:1], ws)
    refused(m.cache.attend, q[:, :3], ws)
    refused(m.cache.attend, q[..., :32], ws)
    refused(m.cache.attend, q.cpu(), ws)
    refused(m.cache.attend, q, ws, out=torch.zeros_like(q)[:, :2])
    refused(m.cache.attend, q, ws, out=torch.zeros_like(q[:, :1]).expand(-1, 4, -1))
    refused(m.cache.attend, q, ws, out=torch.zeros_like(q, dtype=torch.float32))
    refused(m.cache.attend, q, ws, window=-1)
    refused(m.cache.attend, q, ws, sinks=-2)
    refused(m.cache.attend, q, ws, lse=new(torch.zeros, 2, 3))
    refused(m.cache.attend, q, ws, mass=new(torch.zeros, 2, 1, 40))
    refused(m.cache.attend, q, ws, mass=new(torch.zeros, 2, 2, 40, dtype=torch.float64))
    refused(m.cache.attend, q, ws, mass=new(torch.zeros, 2, 2, 40), mass_out=new(torch.zeros, 2, 2, 41))
    big = new(torch.zeros, 2, 2, 90)
    refused(m.cache.attend, q, ws, mass=big[..., :40], mass_out=big[..., 1:41])      # overlapping, not equal
    # a workspace without room for the mass
    refused(m.cache.attend, q, ws, out=torch.zeros_like(q), mass=new(torch.zeros, 2, 2, 32))
    refused(m.cache.attend, q.clone().requires_grad_(), ws)
    with torch.no_grad():
        runs(m.cache.attend, q.clone().requires_grad_(), ws, out=torch.zeros_like(q))


def budgets(new, to_gpu, runs):
    m = to_gpu(R.make([20, 3], 2, 64, 16, torch.bfloat16, heads=4, seed=1))
    mass = new(torch.rand, 2, 2, 32)
    refused(m.cache.evict, mass, 0)
    refused(m.cache.evict, mass, 8, sinks=5, recent=4)
    refused(m.cache.evict, mass, 8, sinks=-1)
    refused(m.cache.evict, mass[:1], 8)
    refused(m.cache.evict, None, 8)
    refused(m.cache.evict, mass, 8, kept=new(torch.zeros, 2, 2, 9, dtype=torch.int32))
    refused(m.cache.evict, mass, 8, kept=new(torch.zeros, 2, 2, 8))
    other = to_gpu(R.make([8], 2, 64, 16, torch.bfloat16, seed=2))
    refused(m.cache.evict, mass, 8, to=other.cache)
    small = to_gpu(R.make([8, 3], 2, 64, 4, torch.bfloat16, seed=2))
    refused(m.cache.evict, mass, 20, to=small.cache)
    # a destination over the same pools with another table could write what is still to be read
    refused(m.cache.evict, mass, 8, to=S.KVCache(m.gk, m.gv, m.gtable.clone(), m.glens.clone()),
            kept=new(torch.zeros, 2, 2, 8, dtype=torch.int32))
