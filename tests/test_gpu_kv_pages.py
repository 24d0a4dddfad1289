"""Who has which pages of a cache: count, fork, resize, compact and copy against
the plain reference, in walks of many steps."""
import random

import pytest
import torch

import lossless_bf16_tensor_splitzip_amd as S
from kv_pages_reference import BAD_LEN, BAD_PAGE, BAD_PARENT, NO_PAGE, Pool
from test_gpu_parity import DEV, _say

pytestmark = pytest.mark.gpu


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Made:
    """A pool on the GPU and its reference; pages of every sequence in random order."""

    def __init__(self, lens, pages, page, width, layers=1, kv_heads=1, dim=8, layout="hnd", dtype=torch.bfloat16, seed=0):
        rng = random.Random(seed)
        g = torch.Generator().manual_seed(seed)
        self.page, self.width = page, width
        free = list(range(pages))
        rng.shuffle(free)
        table = [[free.pop() if i < -(-n // page) else -1 for i in range(width)] for n in lens]
        shape = (layers, 2, pages, kv_heads, page, dim) if layout == "hnd" else (layers, 2, pages, page, kv_heads, dim)
        kv = torch.randint(-30000, 30000, shape, generator=g, dtype=torch.int16).view(dtype)
        if layout == "nhd":
            kv = kv.transpose(3, 4)
        self.ref = Pool(table, lens, kv.clone(), page)
        self.kv = torch.empty_strided(kv.shape, kv.stride(), dtype=dtype, device=DEV).copy_(kv)
        self.table = torch.tensor(table, dtype=torch.int32, device=DEV).reshape(len(lens), width)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.caches = [S.KVCache(k, v, self.table, self.lens) for k, v in self.kv]
        self.pages = S.KVPages(self.caches)
        self.pages.state.fill_(0x5A)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.moved = torch.full((pages,), -7, dtype=torch.int32, device=DEV)

    def check(self, what=""):
        torch.cuda.synchronize()
        assert int(self.status) == self.ref.status, what
        assert self.lens.tolist() == self.ref.lens, what
        assert self.table.tolist() == self.ref.table, what
        assert self.pages.refs.tolist() == self.ref.refs(), what
        assert torch.equal(self.kv.cpu().contiguous().view(torch.int16), self.ref.kv.contiguous().view(torch.int16)), what

    def count(self):
        self.pages.count(status=self.status)
        self.ref.count()

    def fork(self, parents):
        self.pages.fork(ints(parents), status=self.status)
        self.ref.fork(parents)

    def resize(self, lens):
        self.pages.resize(ints(lens), status=self.status)
        self.ref.resize(lens)

    def compact(self):
        used = self.pages.compact(moved=self.moved, status=self.status)
        want, moved = self.ref.compact()
        assert int(used) == want
        assert self.moved.tolist() == moved


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def walk(m, steps, rng, most):
    m.count()
    m.check("count")
    batch = len(m.ref.lens)
    for step in range(steps):
        kind = rng.choice(["fork", "grow", "grow", "grow", "any", "compact", "end"])
        if kind == "fork":
            m.fork([rng.choice([b, b, rng.randrange(batch)]) for b in range(batch)])
        elif kind == "end":
            m.fork([b if rng.random() < 0.7 else -1 for b in range(batch)])
        elif kind == "grow":
            more = rng.choice([1, 1, 5, 40])
            m.resize([min(most, n + (rng.random() < 0.8) * more) for n in m.ref.lens])
        elif kind == "any":
            m.resize([rng.choice([n, rng.randint(0, most)]) for n in m.ref.lens])
        else:
            m.compact()
        m.check("%d %s" % (step, kind))


@pytest.mark.parametrize("page", [1, 3, 16, 64])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
@pytest.mark.parametrize("batch", [1, 5, 33])
def test_walks(batch, layout, page):
    """Pools that mostly suffice and sometimes run out."""
    _say("pages walk batch=%d %s page=%d" % (batch, layout, page))
    rng = random.Random(batch * 100 + page)
    most = 150
    lens = [rng.choice([0, 1, rng.randint(0, most)]) for _ in range(batch)]
    held = sum(-(-n // page) for n in lens)
    dim, kv_heads = rng.choice([(8, 1), (64, 2), (40, 3)])
    m = Made(lens, held + 40 + batch * (most // page) // 3, page, -(-most // page), layers=rng.choice([1, 2, 3]),
             kv_heads=kv_heads, dim=dim, layout=layout, seed=batch + page)
    walk(m, 25, rng, most)


def test_many_layers():
    """More pools than one launch moves pages of."""
    _say("pages of 70 layers")
    m = Made([20, 7, 0], 30, 8, 6, layers=70, kv_heads=2, dim=16, layout="nhd", seed=5)
    m.count()
    m.fork([0, 0, 0])
    m.check()
    m.resize([21, 24, 47])
    m.check()
    m.fork([-1, 1, 2])
    m.compact()
    m.check()


@pytest.mark.parametrize("batch,width", [(300, 130), (1025, 70), (5000, 3), (17000, 2), (65535, 1)])
def test_wide_batches(batch, width):
    """Every form of the fork, and sequences in several rounds of the choice."""
    _say("pages of %d sequences" % batch)
    rng = random.Random(batch)
    lens = [rng.randint(0, width * 2) for _ in range(batch)]
    m = Made(lens, sum(-(-n // 2) for n in lens) + batch, 2, width, seed=batch)
    m.count()
    m.check("count")
    m.fork([rng.choice([b, rng.randrange(batch), rng.randrange(3), -1]) for b in range(batch)])
    m.check("fork")
    m.resize([rng.randint(0, width * 2) for _ in range(batch)])
    m.check("resize")
    m.resize([min(width * 2, n + 1) for n in m.ref.lens])
    m.check("one more")
    m.compact()
    m.check("compact")


def test_large_pool():
    """More blocks of pages than the choice looks at in one round, most of them full."""
    _say("a pool of 600000 pages")
    rng = random.Random(1)
    pages, width = 600_001, 150_000
    m = Made([width, width, width, width - 7, 0], pages, 1, width, seed=3)
    m.count()
    m.check("count")
    m.resize([0, width, width - 1000, width, 1000])
    m.check("resize")
    m.compact()
    m.check("compact")
    m.resize([width, 5, width, width, width])
    m.check("runs out")               # 600005 pages asked for
    m.resize([width] * 5)
    m.check("runs out")
    assert m.ref.status == NO_PAGE


def test_a_full_pool():
    """No page for a copy, none for an entry, in order of the sequences."""
    _say("pages run out")
    m = Made([20, 3, 16, 0], 6, 8, 8, layers=2, kv_heads=2, dim=16)
    m.count()
    m.fork([0, 0, 2, 3])              # 0 and 1 share 3 pages, 2 has 2: one is left
    m.check()
    m.resize([24, 25, 16, 1])         # 1's copy takes it, its fourth page and 3's first are not there
    m.check()
    assert m.ref.lens == [24, 24, 16, 0] and m.ref.status == NO_PAGE
    m.resize([64, 0, 0, 0])           # what the others free is taken by the first
    m.check()
    assert m.ref.lens == [48, 0, 0, 0]
    m.resize([17, 0, 0, 0])
    m.fork([0, 0, 0, 0])
    m.resize([48, 17, 18, 18])        # three of the four write the shared page: all copy it, first come
    m.check()


def test_who_keeps_a_shared_page():
    """All that name it write it: the first keeps it; one does not: all copy."""
    for parents, lens in (([0, 0, 0], [6, 6, 6]), ([0, 0, 0], [5, 6, 6]), ([0, 0, 2], [6, 5, 9]), ([0, 0, 0], [5, 5, 6]),
                          ([0, 0, 0], [4, 6, 6]), ([0, 0, 0], [0, 6, 5]), ([0, 0, 0], [16, 16, 3])):
        m = Made([5, 1, 2], 12, 4, 4, layers=2, kv_heads=3, dim=8, layout="nhd")
        m.count()
        m.fork(parents)
        m.resize(lens)
        m.check((parents, lens))


@pytest.mark.parametrize("lens,want", [
    # pages of 4; 0, 1 and 2 share one with 3, 1 and 2 slots in use; `spare` pages are free
    ((0, [4, 2, 3]), [3, 1, 2]),          # no copy to be had: nobody may write the page
    ((1, [4, 2, 3]), [3, 2, 2]),          # one has its own
    ((2, [4, 2, 3]), [4, 2, 3]),          # the first keeps it
    ((2, [8, 2, 3]), [3, 2, 2]),          # its own next page leaves one copy: it gets neither page nor length
    ((3, [8, 2, 3]), [8, 2, 3]),
    ((0, [4, 1, 0]), [3, 1, 0]),          # 1 reads it: 0 must copy
    ((0, [4, 0, 0]), [4, 0, 0]),          # nobody else names it
])
@pytest.mark.parametrize("far", [0, 1100])
def test_the_page_that_is_kept_when_pages_run_out(lens, want, far):
    """The sequence that would keep the page it shares does not write over one that has no copy."""
    _say("a kept page, %s, %d sequences between" % (lens, far))
    spare, lens = lens
    between = [0] * far
    m = Made([3] + between + [0, 0], 1 + spare, 4, 2, layers=2, kv_heads=2)
    m.count()
    m.fork([0] + list(range(1, far + 1)) + [0, 0])
    m.resize([3] + between + [1, 2])
    m.check("shared")
    m.resize([lens[0]] + between + lens[1:])
    m.check((lens, far))
    got = m.lens.tolist()
    assert [got[0]] + got[far + 1:] == want


def test_findings():
    """What only the device sees: left out, reported."""
    _say("findings of the page operators")
    m = Made([20, 3, 16], 12, 8, 4)
    m.table[0, 1] = 12
    m.table[2, 0] = -5
    m.ref.table[0][1], m.ref.table[2][0] = 12, -5
    m.count()
    m.check("count")
    assert m.ref.status == BAD_PAGE
    m.fork([3, -2, 2])
    m.check("parents")
    assert m.ref.status == BAD_PAGE | BAD_PARENT
    m.resize([20, 33, -1])
    m.check("lengths")
    assert m.ref.status == BAD_PAGE | BAD_PARENT | BAD_LEN
    # tokens that the table has no page for: a page, reported, no copy
    m = Made([9, 3, 16], 12, 8, 4)
    m.table[0, 1] = -1
    m.ref.table[0][1] = -1
    m.count()
    m.resize([10, 3, 16])
    m.check("missing")
    assert m.ref.status == BAD_PAGE


def test_resize_to_its_own_lengths():
    """After lengths were cut by others, their pages go."""
    m = Made([20, 3, 16], 12, 8, 4)
    m.count()
    m.lens.copy_(ints([9, 0, 16]))
    m.ref.lens = [9, 0, 16]
    m.pages.resize(m.lens, status=m.status)
    m.ref.resize([9, 0, 16])
    m.check()
    assert m.pages.refs.sum().item() == 4


@pytest.mark.parametrize("layouts", [("hnd", "hnd"), ("nhd", "nhd"), ("hnd", "nhd"), ("nhd", "hnd")])
@pytest.mark.parametrize("kv_heads,page,dim", [(1, 1, 8), (3, 16, 64), (8, 24, 80), (1, 7, 256), (16, 1, 128), (5, 64, 8)])
def test_copy(layouts, kv_heads, page, dim):
    _say("copy pages %s %d %d %d" % (layouts, kv_heads, page, dim))
    a = Made([], 40, page, 0, layers=3, kv_heads=kv_heads, dim=dim, layout=layouts[0], dtype=torch.float16, seed=1)
    b = Made([], 31, page, 0, layers=3, kv_heads=kv_heads, dim=dim, layout=layouts[1], dtype=torch.float16, seed=2)
    rng = random.Random(page)
    src = [rng.randrange(40) for _ in range(20)]          # a page may be read twice
    dst = rng.sample(range(31), 20)
    src[3], dst[7] = 40, -1
    a.pages.copy(ints(src), ints(dst), to=b.pages, status=a.status)
    a.ref.copy(src, dst, b.ref)
    both = rng.sample(range(40), 24)
    a.pages.copy(ints(both[:12]), ints(both[12:]), status=a.status)
    a.ref.copy(both[:12], both[12:], a.ref)
    a.pages.copy(ints([]), ints([]), to=b.pages)
    torch.cuda.synchronize()
    assert int(a.status) == BAD_PAGE == a.ref.status
    for m in (a, b):
        assert torch.equal(m.kv.cpu().contiguous().view(torch.int16), m.ref.kv.contiguous().view(torch.int16))
