"""Lengths that change in the caches between two calls of the page operators (an
eviction in place, tokens taken back, lens += 1): whatever a fork has shared
before, ``resize`` leaves no page that a sequence is about to write to another."""
import random

import pytest
import torch

import lossless_bf16_tensor_splitzip_amd as S
import kv_reference as R
from kv_pages_reference import BAD_PAGE, NO_PAGE, Pool
from test_gpu_kv_pages import Made, ints
from test_gpu_parity import DEV, _say

pytestmark = pytest.mark.gpu


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Cut(Pool):
    """A resize frees what lies behind the length in the cache, too, and a sequence grows from that length or from the
    one that the last call left."""

    def count(self):
        super().count()
        self.left = list(self.lens)

    def fork(self, parents):
        super().fork(parents)
        self.left = list(self.lens)

    def resize(self, lens):
        most = len(self.table[0]) * self.page
        now, old = self.lens, [min(n, was) for n, was in zip(self.lens, self.left)]
        for row, was, n in zip(self.table, now, lens):
            keep = self.need(min(was, max(n, 0), most))
            row[keep:] = [-1] * (len(row) - keep)
        before = [list(row) for row in self.table]
        self.lens = list(old)
        super().resize(lens)
        refs = self.refs()
        for row, had, was, long, n in zip(self.table, before, old, now, self.lens):
            at = was // self.page
            if n <= was:
                continue
            assert all(refs[p] == 1 for p in row[at:self.need(n)])       # what will be written is one sequence's
            if was % self.page and row[at] != had[at]:                  # all that the cache says is in use
                slots = min(long - at * self.page, self.page)
                self.kv[:, :, row[at], :, :slots] = self.kv[:, :, had[at], :, :slots]
        self.left = list(self.lens)


def made(*args, **kw):
    m = Made(*args, **kw)
    m.ref.__class__ = Cut
    m.count()
    return m


def set_lens(m, lens):
    m.lens.copy_(ints(lens))
    m.ref.lens = list(lens)


# `far` sequences of no tokens between the others: more than one workgroup plans
@pytest.mark.parametrize("far", [0, 1100])
@pytest.mark.parametrize("cut,grown", [(20, 36), (16, 17), (17, 18), (0, 1), (0, 40), (32, 48), (31, 33), (40, 41)])
def test_cut_forked_grown(cut, grown, far):
    _say("cut to %d, forked, grown to %d, %d sequences between" % (cut, grown, far))
    between = [0] * far
    m = made([40] + between + [0], 12, 16, 3, layers=2, kv_heads=2)
    set_lens(m, [cut] + between + [0])
    m.fork([0] + list(range(1, far + 1)) + [0])
    m.check("forked")
    m.resize([grown] + between + [grown])
    m.check("grown")
    assert m.ref.status == 0


@pytest.mark.parametrize("far", [0, 1100])
@pytest.mark.parametrize("cut,grown", [(32, 33), (30, 33), (32, 160), (7, 8), (0, 1), (0, 160), (144, 145), (159, 160)])
def test_forked_cut_grown(cut, grown, far):
    _say("forked, one cut to %d and grown to %d, %d sequences between" % (cut, grown, far))
    between = [0] * far
    m = made([160] + between + [0], 30, 16, 10, layers=2, kv_heads=2)
    m.fork([0] + list(range(1, far + 1)) + [0])
    set_lens(m, [160] + between + [cut])
    m.resize([160] + between + [grown])
    m.check((cut, grown))
    assert m.ref.status == 0


def test_evicted_forked_grown():
    """By an eviction, with the tokens that are appended behind it."""
    _say("evicted in place, forked, grown")
    m = made([40, 0, 25], 14, 16, 3, kv_heads=2, dim=64)
    cache = m.caches[0]
    mass = torch.rand(3, 2, 48, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    cache.evict(mass, 20)
    m.ref.lens = [20, 0, 20]
    m.fork([0, 0, 2])
    m.resize([36, 37, 21])
    torch.cuda.synchronize()
    assert m.lens.tolist() == m.ref.lens and m.table.tolist() == m.ref.table and m.pages.refs.tolist() == m.ref.refs()
    cu = ints([0, 16, 33, 34])
    k = torch.randn(34, 2, 64, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(DEV)
    cache.append(k, -k, cu, status=m.status)
    got, back = torch.zeros_like(k), torch.zeros_like(k)
    cache.gather(got, back, cu, status=m.status)
    torch.cuda.synchronize()
    assert int(m.status) == 0
    assert torch.equal(got, k) and torch.equal(back, -k)


@pytest.mark.parametrize("page", [1, 3, 16])
@pytest.mark.parametrize("batch", [4, 33])
def test_walks_with_cuts(batch, page):
    """Forks, growth and cuts in place in any order; pools that sometimes run out."""
    _say("walk with cuts, batch=%d page=%d" % (batch, page))
    rng = random.Random(batch * 10 + page)
    most = 60
    lens = [rng.randint(0, most) for _ in range(batch)]
    pages = sum(-(-n // page) for n in lens) + 10 + batch * (most // page) // 3
    m = made(lens, pages, page, -(-most // page), layers=2, kv_heads=2, dim=16, layout="nhd", seed=page)
    for step in range(40):
        kind = rng.choice(["fork", "cut", "cut", "grow", "grow", "longer", "longer", "any", "own", "compact"])
        if kind == "fork":
            m.fork([rng.choice([b, b, rng.randrange(batch), -1]) for b in range(batch)])
        elif kind == "cut":
            set_lens(m, [rng.choice([n, max(0, n - rng.choice([1, 5, 30]))]) for n in m.ref.lens])
        elif kind == "grow":
            more = rng.choice([1, 1, 5, 40])
            m.resize([min(most, n + (rng.random() < 0.8) * more) for n in m.ref.lens])
        elif kind == "longer":
            m.ref.lens = list(m.ref.left)
            set_lens(m, [min(most, n + rng.choice([0, 1, 1, 20])) for n in m.ref.lens])
            m.pages.resize(rng.choice([m.lens, m.lens.clone()]), status=m.status)
            m.ref.resize(list(m.ref.lens))
        elif kind == "any":
            m.resize([rng.choice([n, rng.randint(0, most)]) for n in m.ref.lens])
        elif kind == "own":
            m.pages.resize(m.lens, status=m.status)
            m.ref.resize(list(m.ref.lens))
        else:
            m.compact()
        m.check("%d %s" % (step, kind))
    assert m.ref.status in (0, NO_PAGE)


@pytest.mark.parametrize("far", [0, 1100])
@pytest.mark.parametrize("own", [True, False])
@pytest.mark.parametrize("more,ask", [(1, 0), (12, 0), (13, 0), (40, 0), (1, 5), (20, 1), (3, -2)])
def test_made_longer_in_place(more, ask, own, far):
    """lens += 1 comes before the resize: the page that all of them begin is still copied."""
    _say("longer in place by %d, asked for %d more, own=%s, %d sequences between" % (more, ask, own, far))
    between = [0] * far
    m = made([20] + between + [0, 0], 20, 16, 5, layers=2, kv_heads=2)
    m.fork([0] + list(range(1, far + 1)) + [0, 0])
    set_lens(m, [20 + more] + between + [20 + more, 20])
    target = ints([n + ask if n > 20 else n for n in m.ref.lens])
    if own and not ask:
        target = m.lens
    m.ref.resize(target.tolist())
    m.pages.resize(target, status=m.status)
    m.check((more, ask))
    assert m.ref.status == 0 and m.ref.lens == [20 + more + ask] + between + [20 + more + ask, 20]


@pytest.mark.parametrize("lens,want", [([4, 2, 3], [3, 1, 2]), ([3, 2, 2], [3, 1, 2]), ([4, 1, 0], [3, 1, 0])])
def test_longer_in_place_and_no_page(lens, want):
    """A copy that is not to be had: the length that the last call left, not the one that was written into the cache."""
    m = made([3, 0, 0], 1, 4, 1, layers=2, kv_heads=2)
    m.fork([0, 0, 0])
    m.resize([3, 1, 2])
    set_lens(m, lens)
    m.pages.resize(m.lens, status=m.status)
    m.ref.resize(lens)
    m.check(lens)
    assert m.lens.tolist() == want and m.ref.status == NO_PAGE


def test_room_that_is_used_later():
    """Room is made, the length taken back and made longer again as tokens come, without a call; a fork of others, and of
    that sequence, comes between."""
    _say("room that is used later")
    m = made([40, 17, 0], 20, 16, 6, kv_heads=2, dim=64)
    cache, rows = m.caches[0], torch.randn(96, 2, 64, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(DEV)
    m.pages.resize(ints([90, 17, 0]))

    def append(first, last, sequence=0):
        cu = [0] * (sequence + 1) + [last - first] * (3 - sequence)
        cache.lens[sequence] = last
        cache.append(rows[first:last], -rows[first:last], ints(cu), status=m.status)

    def cached(sequence, n):
        cu = ints([0] * (sequence + 1) + [n] * (3 - sequence))
        k, v = torch.zeros_like(rows[:n]), torch.zeros_like(rows[:n])
        cache.gather(k, v, cu, start=ints([0, 0, 0]), status=m.status)
        assert torch.equal(k, rows[:n]) and torch.equal(v, -rows[:n])

    append(0, 20)
    append(0, 17, 1)
    m.pages.fork(ints([0, 1, 1]))             # of another
    for last in range(21, 42):
        append(last - 1, last)
    m.pages.resize(ints([42, 17, 18]))        # in use: none of it goes
    append(41, 42)
    append(17, 18, 2)
    cached(0, 42)
    cached(1, 17)
    cached(2, 18)
    m.pages.fork(ints([0, 0, 2]))             # of this one
    m.pages.resize(ints([43, 44, 18]))
    append(42, 43)
    append(42, 44, 1)
    cached(0, 43)
    cached(1, 44)
    cached(2, 18)
    torch.cuda.synchronize()
    assert int(m.status) == 0


@pytest.mark.parametrize("far", [0, 1100])
@pytest.mark.parametrize("gap,width", [((1, 3), 5), ((2, 4), 5), ((1, 70), 100), ((3, 90), 100), ((0, 65), 200)])
def test_rows_with_gaps(gap, width, far):
    """Page numbers outside the pool leave gaps in a row; what is behind them is freed all the same."""
    _say("a row without its entries %d to %d, %d sequences between" % (gap[0], gap[1] - 1, far))
    between, page = [0] * far, 4
    lens = [page * (width - 1)] + between + [7]
    m = Made(lens, 2 * width + 5, page, width, layers=2)
    m.ref.__class__ = Cut
    for i in range(*gap):
        m.ref.table[0][i] = -1 if i % 2 else 1 << 20
    m.table.copy_(ints(m.ref.table))
    m.count()
    m.check("counted")
    assert m.ref.status == BAD_PAGE
    m.fork([0] + list(range(1, far + 1)) + [0])
    for n in (lens[0] - 1, page * gap[1] + 2, page * gap[0] + 1, page * gap[0] + 3, page, 1, 0, 2 * page + 1):
        m.resize([n] + between + [max(0, n - 3)])
        m.check(n)
    m.count()
    assert sum(m.ref.refs()) == m.ref.need(2 * page + 1) + m.ref.need(2 * page - 2)
    m.check("counted again")


def test_layers_evicted():
    """In place, one layer after another with the lengths of before; then the pages behind are free, and the samples of a
    sequence go on in pages of their own."""
    _say("layers evicted in place")
    lens, budget, kvh, dim = [90, 33, 50, 0], 40, 2, 64
    m = made(lens, 24, 16, 6, layers=3, kv_heads=kvh, dim=dim)
    gen = torch.Generator().manual_seed(4)
    old, masses = m.ref.kv.clone(), [torch.rand(4, kvh, 96, generator=gen) for _ in m.caches]
    table = [list(r) for r in m.ref.table]
    before = m.lens.clone()
    for c, mass in zip(m.caches, masses):
        m.lens.copy_(before)
        c.evict(mass.to(DEV), budget, sinks=2, recent=5, status=m.status)
    short = [min(n, budget) for n in lens]
    m.pages.resize(m.lens, status=m.status)
    m.pages.fork(ints([0, 1, 2, 0]), status=m.status)
    m.pages.resize(ints([41, 33, 40, 47]), status=m.status)
    torch.cuda.synchronize()
    assert int(m.status) == 0
    assert m.pages.refs.sum().item() == sum(m.ref.need(n) for n in [41, 33, 40, 47])
    now, kv = m.table.tolist(), m.kv.cpu()
    for i, mass in enumerate(masses):
        for b, parent in enumerate([0, 1, 2, 0]):
            n = lens[parent]
            for h in range(kvh):
                kept = R.evict(mass[parent, h], n, budget, 2, 5) if n > budget else range(n)
                assert len(kept) == short[parent]
                for to, t in enumerate(kept):
                    want = old[i, :, table[parent][t // 16], h, t % 16]
                    got = kv[i, :, now[b][to // 16], h, to % 16]
                    assert torch.equal(want.view(torch.int16), got.view(torch.int16)), (i, b, h, to)


@pytest.mark.parametrize("batch,width", [(300, 130), (1025, 70), (5000, 3), (17000, 2), (65535, 1)])
def test_wide_batches_cut_and_made_longer(batch, width):
    """Every form of the count, the fork and the choice keeps the lengths that it left."""
    _say("lengths of %d sequences" % batch)
    rng = random.Random(batch)
    page, most = 3, 3 * width
    lens = [rng.randint(0, most) for _ in range(batch)]
    m = made(lens, sum(-(-n // page) for n in lens) + 3 * batch, page, width, seed=batch)
    for turn in range(3):
        if turn:
            m.fork([rng.choice([b, rng.randrange(batch), rng.randrange(3)]) for b in range(batch)])
        longer = turn != 1
        set_lens(m, [min(most, n + rng.randrange(3)) if longer else rng.randint(0, n) for n in m.ref.lens])
        m.pages.resize(m.lens, status=m.status)
        m.ref.resize(list(m.ref.lens))
        m.check(("itself", turn))
        m.resize([min(most, n + 1) for n in m.ref.lens])
        m.check(("one more", turn))
    assert m.ref.status == 0
