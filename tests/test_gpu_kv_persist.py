"""The cache and the codec together: a sequence leaves the GPU as payloads and
comes back bit for bit, and a few steps of serving around it."""
import pytest
import torch

import lossless_bf16_tensor_splitzip_amd as S
import kv_reference as R
import workloads as W
from test_gpu_parity import DEV

pytestmark = pytest.mark.gpu


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def bits(t):
    return t.contiguous().view(torch.int16)


@pytest.mark.parametrize("n", [0, 1, 333])
def test_a_sequence_leaves_and_returns(n):
    m = R.to_gpu(R.make([40, n, 7], 4, 128, 16, torch.bfloat16, seed=n, slack=30), S)
    ws = S.Workspace(max(n, 1) * 4 * 128, DEV)
    packed = S.persist.pack_sequence("layer.0", m.cache, 1, ws)
    assert packed[0][0]["name"] == "layer.0.k" and packed[1][0]["shape"] == [4, n, 128]
    if n > 1:
        assert packed[0][1].numel() < 0.8 * 2 * n * 4 * 128
    # into other pages of the same pools
    used = set(m.table[m.table >= 0].tolist())
    free = [p for p in range(m.k.shape[0]) if p not in used]
    need = -(-n // 16)
    old_k, old_v = (R.rows(m, 1, torch.arange(n), pool) for pool in (m.k, m.v))
    m.table[1, :need] = torch.tensor(free[:need], dtype=torch.int32)
    m.gtable.copy_(m.table)
    m.glens[1] = 0
    assert S.persist.unpack_sequence(packed, m.cache, 1) == n
    assert int(m.glens[1]) == n
    for pool, old in ((m.gk, old_k), (m.gv, old_v)):
        assert torch.equal(bits(R.rows(m, 1, torch.arange(n), pool.cpu())), bits(old))


def test_misfits_are_refused():
    m = R.to_gpu(R.make([40, 20], 4, 128, 16, torch.bfloat16, seed=3), S)
    ws = S.Workspace(40 * 4 * 128, DEV)
    packed = S.persist.pack_sequence("x", m.cache, 0, ws)
    other = R.to_gpu(R.make([40], 2, 128, 16, torch.bfloat16, seed=3), S)
    small = R.to_gpu(R.make([30], 4, 128, 8, torch.bfloat16, seed=3, width=4), S)
    for cache, b in ((other.cache, 0), (small.cache, 0), (m.cache, 2), (m.cache, -1)):
        with pytest.raises(ValueError):
            S.persist.unpack_sequence(packed, cache, b)
    with pytest.raises(ValueError):
        S.persist.pack_sequence("x", m.cache, 2, ws)
    m.gtable[0, 2] = -1
    with pytest.raises(ValueError):
        S.persist.pack_sequence("x", m.cache, 0, ws)


def test_serving_steps():
    """Prompts arrive as payloads, tokens are generated with windowless
    attention that keeps the mass, and the cache is evicted whenever it passes
    its budget: K and V, mass and outputs follow a plain model of the cache."""
    heads, kv_heads, dim, page, budget = 8, 2, 64, 16, 96
    lens = [90, 20, 0]
    m = R.make(lens, kv_heads, dim, page, torch.bfloat16, seed=5, fill=0.0, width=8, slack=24, heads=heads)
    used = set(m.table[m.table >= 0].tolist())
    free = [p for p in range(m.k.shape[0]) if p not in used]
    for b in range(3):
        for j in range(8):
            if m.table[b, j] < 0:
                m.table[b, j] = free.pop()
    prompts = [(R.rows(m, b, torch.arange(n), m.k), R.rows(m, b, torch.arange(n), m.v)) for b, n in enumerate(lens)]
    R.to_gpu(m, S)
    cache = m.cache
    ws = S.Workspace(kv_heads * 128 * dim, DEV)
    for b, n in enumerate(lens):        # through the codec, as a transfer would bring them
        packed = S.persist.pack_sequence("prompt", cache, b, ws)
        m.gk[m.gtable[b].long()], m.gv[m.gtable[b].long()] = 0, 0
        S.persist.unpack_sequence(packed, cache, b)
    # the plain model: per sequence and head, rows of K, V and mass
    plain = [[[prompts[b][0][:, h].clone(), prompts[b][1][:, h].clone(), torch.zeros(n, dtype=torch.float64)]
              for h in range(kv_heads)] for b, n in enumerate(lens)]
    mass = torch.zeros(3, kv_heads, 128, device=DEV)
    kws = S.KVWorkspace(cache, heads, mass=True)
    cu = torch.tensor([0, 1, 2, 2], dtype=torch.int32, device=DEV)       # the third slot of the batch stays empty
    evictions = 0
    for step in range(14):
        q, k, v = (W.to_bf16(W.normal(3 * c * dim, 40, 10 * step + i)).reshape(3, c, dim)
                   for i, c in enumerate((heads, kv_heads, kv_heads)))
        m.glens.add_(torch.tensor([1, 1, 0], dtype=torch.int32, device=DEV))
        cache.append(k[:2].to(DEV), v[:2].to(DEV), cu)
        out = cache.attend(q.to(DEV), kws, mass=mass).double().cpu()
        assert bool((out[2] == 0).all())
        for b in range(2):
            for h in range(kv_heads):
                pk, pv, pm = plain[b][h]
                pk, pv = torch.cat([pk, k[b, h][None]]), torch.cat([pv, v[b, h][None]])
                pm = torch.cat([pm, torch.zeros(1, dtype=torch.float64)])
                for i in range(h * 4, h * 4 + 4):
                    p = torch.softmax(pk.double() @ q[b, i].double() * dim ** -0.5, 0)
                    want = p @ pv.double()
                    tol = 2.0 ** -8 * want.abs() + 2.0 ** -12 * (p @ pv.double().abs())
                    assert bool(((out[b, i] - want).abs() <= tol).all()), (step, b, i)
                    pm = pm + p
                plain[b][h] = [pk, pv, pm]
                got = mass[b, h, :pm.numel()].double().cpu()
                assert bool(((got - pm).abs() <= 2.0 ** -16 * (step + 1)).all()), (step, b, h)
        if int(m.glens.max()) > budget:
            evictions += 1
            now = mass.cpu()
            cache.evict(mass, budget - 4, sinks=4, recent=16)
            for b in range(2):
                for h in range(kv_heads):
                    pk, pv, pm = plain[b][h]
                    keep = R.evict(now[b, h], pm.numel(), budget - 4, 4, 16)
                    plain[b][h] = [pk[keep], pv[keep], now[b, h, keep].double()]
            assert m.glens.tolist() == [plain[0][0][0].shape[0], plain[1][0][0].shape[0], 0]
    assert evictions >= 2
    m.table = m.gtable.cpu()
    for b in range(2):
        n = int(m.glens[b])
        for h in range(kv_heads):
            for pool, want in ((m.gk, plain[b][h][0]), (m.gv, plain[b][h][1])):
                assert torch.equal(bits(R.rows(m, b, torch.arange(n), pool.cpu())[:, h]), bits(want))
