"""More of what the tensor-level calls of the key-value cache refuse: tensors
that meet in memory, and those of forward mode.  Written like kv_checks, for a run without a GPU and one
with it."""
import torch
from torch.autograd import forward_ad

import lossless_bf16_tensor_splitzip_amd as S
import kv_reference as R
from kv_checks import refused


def tables(new, to_gpu, runs):
    """Rows of the page table that are one row, or reach into the next: the
    batch * max_pages numbers from its start are not there."""
    m = to_gpu(R.make([20, 3], 2, 64, 16, torch.bfloat16, seed=1))
    k, v, t, n = m.gk, m.gv, m.gtable, m.glens
    refused(S.KVCache, k, v, t[:1].expand(2, -1), n)
    refused(S.KVCache, k, v, t[:1, :1].expand(2, 1), n)
    refused(S.KVCache, k, v, new(torch.zeros, 4, dtype=torch.int32).unfold(0, 3, 1), n)
    wide = new(torch.zeros, 3, 5, dtype=torch.int32)
    assert S.KVCache(k, v, wide[:2, :3], n).args.table_stride == 5          # rows apart
    assert S.KVCache(k, v, wide[:1].expand(1, -1), n[:1]).batch == 1        # one row
    assert S.KVCache(k, v, wide[:1, :0].expand(2, 0), n).max_pages == 0     # rows of nothing


def destinations(new, to_gpu, runs):
    """Evictions into memory that is still to be read."""
    m = to_gpu(R.make([20, 3], 2, 64, 16, torch.bfloat16, seed=1, width=2, slack=6))
    k, v, t, n = m.gk, m.gv, m.gtable, m.glens
    mass = new(torch.rand, 2, 2, 32)
    kept = new(torch.zeros, 2, 2, 8, dtype=torch.int32)
    far = to_gpu(R.make([8, 8], 2, 64, 16, torch.bfloat16, seed=2))
    lens = new(torch.zeros, 3, dtype=torch.int32)
    apart = S.KVCache(k, v, t, lens[:2])

    def into(cache, *to):
        refused(cache.evict, mass, 8, to=S.KVCache(*to), kept=kept)

    into(m.cache, k[1:], v[1:].clone(), far.gtable, far.glens)
    into(m.cache, v[1:], k[1:], far.gtable, far.glens)
    into(apart, far.gk, far.gv, far.gtable, lens[1:])
    # K and V, and the two caches, as slices of one tensor: they interleave and do not meet
    both = new(torch.zeros, 6, 4, 2, 16, 64, dtype=torch.bfloat16)
    one = S.KVCache(both[:, 0], both[:, 1], t, n)
    other = S.KVCache(both[:, 2], both[:, 3], far.gtable, far.glens)
    t.copy_(torch.arange(4, dtype=torch.int32).reshape(2, 2))
    far.gtable.copy_(torch.tensor([[4], [5]], dtype=torch.int32))
    runs(one.evict, mass, 8, to=other, kept=kept)
    runs(one.evict, mass, 8, to=S.KVCache(both[:, 0], both[:, 1], t, n), kept=kept)      # in place


def outputs(new, to_gpu, runs):
    """Outputs that overlap the queries without being the same."""
    m = to_gpu(R.make([20, 3], 2, 64, 16, torch.bfloat16, heads=4, seed=1))
    ws = S.KVWorkspace(m.cache, 4)
    packed = new(torch.zeros, 3, 8, 64, dtype=torch.bfloat16)
    q = packed[:2, :4]
    refused(m.cache.attend, q, ws, out=packed[1:, :4])
    refused(m.cache.attend, q, ws, out=packed[:2, 2:6])
    refused(m.cache.attend, q, ws, out=packed.view(-1)[:512].view(4, 2, 64).transpose(0, 1))
    runs(m.cache.attend, q, ws, out=packed[:2, 4:])              # beside them
    runs(m.cache.attend, q, ws, out=packed[:2, :4])              # in their place
    one = to_gpu(R.make([20], 2, 64, 16, torch.bfloat16, heads=4, seed=1))
    q = packed[:1, :4]                                           # of one sequence, whatever its stride
    runs(one.cache.attend, q, S.KVWorkspace(one.cache, 4), out=q.as_strided((1, 4, 64), (8, 64, 1)))


def gathered(new, to_gpu, runs):
    """Rows of K and V gathered into each other."""
    m = to_gpu(R.make([20, 3], 2, 64, 16, torch.bfloat16, seed=1))
    cu = new(torch.tensor, [0, 2, 4], dtype=torch.int32)
    rows = new(torch.zeros, 6, 4, 64, dtype=torch.bfloat16)
    refused(m.cache.gather, rows[:4, :2], rows[:4, :2], cu)
    refused(m.cache.gather, rows[:4, :2], rows[1:5, 1:3], cu)
    refused(m.cache.gather, rows[:4, 2:], rows[2:, 2:], cu)
    runs(m.cache.gather, rows[:4, :2], rows[:4, 2:], cu)         # halves of the same rows
    runs(m.cache.append, rows[:4, :2], rows[:4, :2], cu)         # read, they may be the same


def pools(new, to_gpu, runs):
    """Pools of K and V that share memory: read, and written where both get
    the same; an eviction in place would move their rows twice."""
    m = to_gpu(R.make([20, 3], 2, 64, 16, torch.bfloat16, heads=4, seed=1))
    far = to_gpu(R.make([8, 3], 2, 64, 16, torch.bfloat16, seed=2))
    k, t, n = m.gk, m.gtable, m.glens
    one, half = S.KVCache(k, k, t, n), S.KVCache(k[:-1], k[1:], t, n)
    cu = new(torch.tensor, [0, 2, 4], dtype=torch.int32)
    rows = new(torch.zeros, 2, 4, 2, 64, dtype=torch.bfloat16)
    mass, kept = new(torch.rand, 2, 2, 32), new(torch.zeros, 2, 2, 8, dtype=torch.int32)
    runs(one.attend, m.gq, S.KVWorkspace(one, 4), out=torch.zeros_like(m.gq))
    runs(one.gather, rows[0], rows[1], cu)
    runs(one.append, rows[0], rows[0], cu)
    runs(one.append, rows[0, :1], rows[0, :1].as_strided((1, 2, 64), (8, 64, 1)), cu)
    refused(one.append, rows[0], rows[1], cu)
    refused(half.append, rows[0], rows[0], cu)
    refused(one.evict, mass, 8, kept=kept)
    refused(half.evict, mass, 8, kept=kept)
    to = S.KVCache(far.gk, far.gk, far.gtable, far.glens)
    refused(m.cache.evict, mass, 8, to=to, kept=kept)
    runs(one.evict, mass, 8, to=to, kept=kept)
    runs(half.evict, mass, 8, to=far.cache, kept=kept)


def masses(new, to_gpu, runs):
    """A mass and its output as slices of one tensor."""
    m = to_gpu(R.make([20, 3], 2, 64, 16, torch.bfloat16, heads=4, seed=1))
    ws = S.KVWorkspace(m.cache, 4, mass=True)
    out, kept = torch.zeros_like(m.gq), new(torch.zeros, 2, 2, 8, dtype=torch.int32)
    both = new(torch.zeros, 2, 4, 80)
    for a, b in ((both[:, :2, :40], both[:, :2, 40:]), (both[:, ::2, :32], both[:, 1::2, :32])):
        runs(m.cache.attend, m.gq, ws, out=out, mass=a, mass_out=b)
        runs(m.cache.evict, a, 8, kept=kept, mass_out=b)
    refused(m.cache.attend, m.gq, ws, out=out, mass=both[:, :2, :40], mass_out=both[:, 1:3, :40])
    refused(m.cache.evict, both[:, :2, :40], 8, kept=kept, mass_out=both[:, :2, 39:79])


def tangents(new, to_gpu, runs):
    """Tensors of forward mode: the tangent would be lost without a word."""
    m = to_gpu(R.make([20, 3], 2, 64, 16, torch.bfloat16, heads=4, seed=1))
    ws = S.KVWorkspace(m.cache, 4, mass=True)
    out, kept = torch.zeros_like(m.gq), new(torch.zeros, 2, 2, 8, dtype=torch.int32)
    cu = new(torch.tensor, [0, 2, 4], dtype=torch.int32)
    rows, mass = new(torch.zeros, 4, 2, 64, dtype=torch.bfloat16), new(torch.zeros, 2, 2, 32)
    with forward_ad.dual_level():
        def dual(t):
            return forward_ad.make_dual(t.clone(), torch.ones_like(t))

        refused(m.cache.attend, dual(m.gq), ws, out=out)
        refused(m.cache.attend, m.gq, ws, out=dual(out))
        refused(m.cache.attend, m.gq, ws, out=out, lse=dual(new(torch.zeros, 2, 4)))
        refused(m.cache.attend, m.gq, ws, out=out, mass=dual(mass))
        refused(m.cache.attend, m.gq, ws, out=out, mass=dual(mass), mass_out=mass)
        refused(m.cache.append, dual(rows), rows, cu)
        refused(m.cache.append, rows, dual(rows), cu)
        refused(m.cache.gather, dual(rows), rows.clone(), cu)
        refused(m.cache.evict, dual(mass), 8, kept=kept)
        refused(S.KVCache, dual(m.gk), m.gv, m.gtable, m.glens)
        with torch.no_grad():                                    # which leaves forward mode on
            refused(m.cache.attend, dual(m.gq), ws, out=out)
        runs(m.cache.attend, m.gq, ws, out=out, mass=mass)
        runs(m.cache.append, rows, rows.clone(), cu)
        runs(m.cache.evict, mass, 8, kept=kept)
    runs(m.cache.attend, m.gq, ws, out=out)


PARTS = ("tables", "destinations", "outputs", "gathered", "pools", "masses", "tangents")
