"""Eviction by accumulated attention weight: which tokens stay, and where
their K, V and mass go, against a plain reference; everything is exact."""
import math

import pytest
import torch

import lossless_bf16_tensor_splitzip_amd as S
import kv_reference as R
from test_gpu_parity import DEV, _say

pytestmark = pytest.mark.gpu


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def bits(t):
    return t.contiguous().view(torch.int16)


def masses(kind, batch, kv_heads, width, seed):
    g = torch.Generator().manual_seed(seed)
    m = torch.rand(batch, kv_heads, width, generator=g) ** 6
    if kind == "ties":
        m = torch.round(m * 4) / 4
    elif kind == "equal":
        m = torch.full_like(m, 0.125)
    elif kind == "signs":
        m = torch.randn(batch, kv_heads, width, generator=g)
        m[..., ::7] = 0.0
        m[..., 1::7] = -0.0
    elif kind == "special":
        m[..., ::5], m[..., 1::11], m[..., 2::13], m[..., 3::9] = math.nan, math.inf, -math.inf, 1e-42
    return m


def check(m, mass, budget, sinks, recent, in_place, mass_apart=False, to_page=16, to_layout="hnd"):
    batch, heads = len(m.lens), m.kv_heads
    old_k, old_v = m.gk.cpu(), m.gv.cpu()
    gm = mass.to(DEV)
    keep = [[R.evict(mass[b, h], m.lens[b], budget, sinks, recent) for h in range(heads)] for b in range(batch)]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    if in_place:
        to = m
    else:
        to = R.to_gpu(R.make([min(n, budget) for n in m.lens], heads, m.dim, to_page, m.dtype, layout=to_layout,
                             seed=99, fill=4.0), S)
        to.glens.fill_(-7)
    mass_out = torch.full_like(gm, -3.0) if mass_apart else None
    kept = m.cache.evict(gm, budget, sinks=sinks, recent=recent, to=None if in_place else to.cache,
                         mass_out=mass_out, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    kept, new_k, new_v = kept.cpu(), to.gk.cpu(), to.gv.cpu()
    got_mass = (gm if mass_out is None else mass_out).cpu()
    seen = torch.zeros(new_k.shape[0], new_k.shape[2], dtype=torch.bool)
    for b in range(batch):
        size, n = min(m.lens[b], budget), m.lens[b]
        assert int(to.glens[b]) == size
        pos = torch.arange(size)
        seen[to.table[b].long()[pos // to.page], pos % to.page] = True
        for h in range(heads):
            want = keep[b][h]
            assert kept[b, h, :size].tolist() == want, (b, h)
            assert bool((kept[b, h, size:] == -1).all())
            for old, new in ((old_k, new_k), (old_v, new_v)):
                assert torch.equal(bits(R.rows(to, b, pos, new)[:, h]), bits(R.rows(m, b, want, old)[:, h])), (b, h)
            assert torch.equal(got_mass[b, h, :size].view(torch.int32), mass[b, h, want].view(torch.int32))
            assert bool((got_mass[b, h, size:n] == 0).all())
            rest = mass[b, h, n:] if mass_out is None else torch.full_like(mass[b, h, n:], -3.0)
            assert torch.equal(got_mass[b, h, n:].view(torch.int32), rest.view(torch.int32))
    if not in_place:          # nothing else of the destination was written
        for new in (new_k, new_v):
            assert bool((new.transpose(1, 2)[~seen] == 4.0).all())
        assert torch.equal(bits(m.gk.cpu()), bits(old_k)) and torch.equal(bits(m.gv.cpu()), bits(old_v))


@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "signs", "special"])
@pytest.mark.parametrize("budget,sinks,recent", [(64, 4, 16), (64, 0, 0), (1, 0, 0), (1, 1, 0), (1, 0, 1), (100, 40, 60),
                                                 (299, 2, 3), (300, 4, 4), (5000, 1, 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_choice(kind, budget, sinks, recent, in_place):
    _say("evict %s budget=%d sinks=%d recent=%d in place=%s" % (kind, budget, sinks, recent, in_place))
    lens = [0, 1, 2, 63, 64, 65, 100, 101, 300]
    m = R.to_gpu(R.make(lens, 2, 64, 16, torch.bfloat16, seed=budget), S)
    check(m, masses(kind, len(lens), 2, 310, budget), budget, sinks, recent, in_place)


@pytest.mark.parametrize("dim,kv_heads,page,layout,to_page,to_layout", [
    (128, 8, 16, "nhd", 7, "hnd"), (8, 1, 1, "hnd", 16, "nhd"), (256, 3, 24, "hnd", 64, "nhd"),
    (200, 2, 33, "nhd", 5, "nhd"), (72, 5, 16, "hnd", 16, "hnd"), (96, 2, 128, "nhd", 1, "hnd")])
@pytest.mark.parametrize("in_place", [False, True])
def test_shapes(dim, kv_heads, page, layout, to_page, to_layout, in_place):
    _say("evict dim=%d heads=%d page=%d in place=%s" % (dim, kv_heads, page, in_place))
    lens = [700, 0, 513, 40]
    m = R.to_gpu(R.make(lens, kv_heads, dim, page, torch.float16, layout=layout, seed=dim), S)
    check(m, masses("plain", 4, kv_heads, 700, dim), 256, 3, 9, in_place, mass_apart=dim % 16 == 0, to_page=to_page,
          to_layout=to_layout)


@pytest.mark.parametrize("n,budget", [(9000, 4500), (40000, 39990), (70001, 3)])
@pytest.mark.parametrize("in_place", [False, True])
def test_long(n, budget, in_place):
    _say("evict %d of %d in place=%s" % (budget, n, in_place))
    m = R.to_gpu(R.make([n, n // 2], 1, 64, 64, torch.bfloat16, seed=n), S)
    check(m, masses("ties" if budget == 4500 else "plain", 2, 1, n, n), budget, 1, 2, in_place)


def test_strided_mass_and_short_mass():
    m = R.to_gpu(R.make([90, 80], 2, 64, 16, torch.bfloat16, seed=1), S)
    g = torch.rand(2, 3, 101, device=DEV)
    before = g.cpu()
    kept = m.cache.evict(g[:, 1:, 3:93], 30, sinks=1, recent=2)
    torch.cuda.synchronize()
    for b, n in enumerate((90, 80)):
        for h in range(2):
            assert kept[b, h].tolist() == R.evict(before[b, h + 1, 3:], n, 30, 1, 2)
    assert torch.equal(g[:, 0].cpu(), before[:, 0]) and torch.equal(g[:, :, :3].cpu(), before[:, :, :3])
    assert torch.equal(g[:, :, 93:].cpu(), before[:, :, 93:])
    # a mass shorter than a sequence: the length is cut to it, and reported
    m = R.to_gpu(R.make([90], 1, 64, 16, torch.bfloat16, seed=1), S)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    kept = m.cache.evict(g[:1, :1, :50].clone(), 30, status=status)
    assert int(status) == 2 and kept[0, 0].tolist() == R.evict(before[0, 0], 50, 30, 0, 0)


def test_bad_page_is_left_out():
    m = R.to_gpu(R.make([64], 1, 64, 16, torch.bfloat16, seed=1, fill=2.0), S)
    m.gtable[0, 1] = 1 << 30
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    old = m.gk.cpu()
    kept = m.cache.evict(torch.rand(1, 1, 64, device=DEV), 40, status=status)[0, 0].tolist()
    torch.cuda.synchronize()
    assert int(status) == 1
    new = m.gk.cpu()
    for i, t in enumerate(kept):
        if i // 16 != 1 and t // 16 != 1:
            assert torch.equal(bits(new[m.table[0, i // 16].long(), 0, i % 16]), bits(old[m.table[0, t // 16].long(), 0, t % 16]))


def test_graph_replays_in_place():
    """Captured eviction in place, replayed as the sequences grow past the
    budget again and again."""
    n, budget = 200, 96
    m = R.to_gpu(R.make([n, 50, 120], 2, 64, 16, torch.bfloat16, seed=7), S)
    mass = torch.zeros(3, 2, n, device=DEV)
    kept = torch.empty(3, 2, budget, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.cache.evict(mass, budget, sinks=2, recent=8, kept=kept)
    for rep in range(5):
        lens = [n - rep, 50, 97 + rep]
        m.glens.copy_(torch.tensor(lens, dtype=torch.int32))
        m.gk.copy_(torch.randn(m.gk.shape, device=DEV))
        mass.copy_(torch.rand(3, 2, n))
        old, was = m.gk.cpu(), mass.cpu()
        g.replay()
        torch.cuda.synchronize()
        for b, ln in enumerate(lens):
            size = min(ln, budget)
            assert int(m.glens[b]) == size
            for h in range(2):
                want = R.evict(was[b, h], ln, budget, 2, 8)
                assert kept[b, h, :size].tolist() == want, rep
                got = R.rows(m, b, torch.arange(size), m.gk.cpu())[:, h]
                assert torch.equal(bits(got), bits(R.rows(m, b, want, old)[:, h])), rep
