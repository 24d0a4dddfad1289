"""Attention of one new token over sequences that begin alike, against a 64-bit
reference of every sequence on its own."""
import math
import random

import pytest
import torch

import lossless_bf16_tensor_splitzip_amd as S
import kv_reference as R
import kv_shared_reference as H
from lossless_bf16_tensor_splitzip_amd import _abi
from test_gpu_parity import DEV, _say

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def close(got, want, tol, what):
    """Within the bound, and equal where that is not finite."""
    got = got.double().cpu()
    odd = ~torch.isfinite(want)
    assert torch.equal(got[odd].nan_to_num(7.0), want[odd].nan_to_num(7.0)), what
    assert bool(((got - want).abs() <= tol)[~odd].all()), (what, float(((got - want).abs() - tol)[~odd].max()))


def widen(m):
    """The same cache with a table so wide that k_shared has the tokens in common, which goes by what a table can hold
    (a group of average size needs more than 16 query rows a KV head); False where that is not so."""
    rows = len(m.lens) * m.q.shape[1] // m.kv_heads // max(len(m.shared), 1)
    if rows <= 16 or not m.shared:
        return False
    width = int(161e6 / (4.0 * m.page * m.kv_heads * m.dim * len(m.shared) * ((rows + 31) // 32))) + 1
    m.table = torch.nn.functional.pad(m.table, (0, max(0, width - m.table.shape[1])), value=-1)
    return True


def check(m, scale=None, hidden=(), want_status=0):
    """With few units a KV head, with as many as a join is for, and, where there are enough rows, with many."""
    out = check_one(m, scale, hidden, want_status)
    table = m.table
    if table.shape[1] * m.page <= 640:
        m.table = torch.nn.functional.pad(table, (0, 640 // m.page + 1 - table.shape[1]), value=-1)
        check_one(m, scale, hidden, want_status)
        m.table = table
    if widen(m):
        check_one(m, scale, hidden, want_status)
        m.table = table
    return out


def check_one(m, scale, hidden, want_status):
    heads = m.q.shape[1]
    R.to_gpu(m, S)
    ws = S.KVSharedWorkspace(m.cache, heads, len(m.shared))
    ws.buf.fill_(0xA5)
    lse = torch.full((len(m.lens), heads), 7.0, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full_like(m.gq, 5.0)
    cu, shared = ints(m.cu), ints(m.shared)
    m.cache.attend_shared(m.gq, cu, shared, ws, out=out, scale=scale, lse=lse, status=status)
    again = m.cache.attend_shared(m.gq, cu, shared, ws, scale=scale)
    torch.cuda.synchronize()
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))
    assert int(status) == want_status
    for b, (o, o_tol, e, e_tol) in enumerate(H.attend(m, scale, hidden)):
        close(out[b], o, o_tol, "out %d" % b)
        close(lse[b], e, e_tol, "lse %d" % b)
    return out


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("dim", [8, 64, 72, 80, 96, 128, 136, 192, 200, 256])
@pytest.mark.parametrize("group", [1, 20])
def test_dims(dtype, dim, group):
    """Few query rows a group, and many."""
    _say("shared dim=%d group=%d %s" % (dim, group, dtype))
    check(H.make([(100, [120, 100, 133]), (40, [41, 300])], 2, dim, 16, dtype, 2 * group, seed=dim + group))


@pytest.mark.parametrize("common", [0, 1, 15, 31, 32, 33, 63, 64, 65, 127, 128, 129, 500, 1000])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads", [8, 48])
def test_tokens_in_common(common, dim, heads):
    _say("shared tokens=%d dim=%d heads=%d" % (common, dim, heads))
    check(H.make([(common, [common + 7, common, common + 70])], 2, dim, 16, BF16, heads, seed=common, layout="nhd"))


@pytest.mark.parametrize("group", [1, 2, 3, 16, 33, 63, 64, 65, 100, 127, 128, 129, 130, 200, 257])
def test_groups_of_heads(group):
    """Sequences that fill a row tile, that do not, and heads of one in several."""
    _say("shared query heads of a KV head=%d" % group)
    check(H.make([(70, [75, 70, 71, 99])], 1, 64, 16, FP16, group, seed=group))


@pytest.mark.parametrize("size", [2, 31, 32, 33, 64, 127, 128, 129, 260])
def test_sizes_of_a_group(size):
    _say("shared by %d sequences" % size)
    rng = random.Random(size)
    check(H.make([(90, [90 + rng.randrange(4) for _ in range(size)])], 2, 64, 32, BF16, 2, seed=size))


@pytest.mark.parametrize("page", [1, 7, 24, 64, 128])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
def test_pages(page, layout):
    _say("shared page=%d %s" % (page, layout))
    check(H.make([(150, [160, 150, 151]), (3, [5, 9])], 3, 80, page, BF16, 6, seed=page, layout=layout))


@pytest.mark.parametrize("groups,heads", [(63, 4), (64, 4), (65, 40), (130, 4), (130, 40), (700, 4), (2049, 2)])
def test_many_groups(groups, heads):
    """Several blocks of groups, runs that have several groups; more than one workgroup holds."""
    _say("shared in %d groups" % groups)
    rng = random.Random(groups)
    made = []
    for _ in range(groups):
        common = rng.choice([0, 1, 20, 64, 65, 140])
        made.append((common, [common + rng.randrange(1 if i else 0, 9) for i in range(rng.choice([1, 2, 3]))]))
    check(H.make(made, 2, 64, 16, BF16, heads, seed=groups))


@pytest.mark.parametrize("heads", [8, 40])
def test_members_of_all_kinds(heads):
    """Ended and short sequences, one that ends where the others go on, a group of one and of none,
    tokens in common beyond the first sequence, sequences in no group."""
    _say("shared: members of all kinds")
    m = H.make([(100, [110, 0, 40, 100, 99, 101]), (50, [80]), (64, [0, 70, 64]), (300, [200, 210, 200])], 2, 128, 16, BF16, heads, seed=3)
    check(m)
    m.cu, m.shared = [0, 6, 6, 7, 10, 13], [100, 30, 50, 64, 300]
    check(m)
    m.cu, m.shared = [1, 1], [100]
    check(m)
    m = H.make([(0, [20, 3]), (64, [100, 70]), (0, [9])], 2, 128, 16, BF16, heads, seed=4)
    m.cu, m.shared = [2, 4], [64]                # sequences before and behind the groups
    check(m)
    m.cu, m.shared = [0], []
    check(m)


def test_nothing_cached():
    _say("shared: nothing cached")
    check(H.make([(10, [0, 0]), (0, [0, 1])], 2, 64, 16, FP16, 4))
    m = R.to_gpu(H.make([], 2, 64, 16, FP16, 4), S)
    assert m.cache.attend_shared(m.gq, ints([0]), ints([]), S.KVSharedWorkspace(m.cache, 4)).shape == (0, 4, 64)


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0, 1e-3])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("heads", [8, 40])
def test_scales(scale, dtype, heads):
    _say("shared scale=%g %s heads=%d" % (scale, dtype, heads))
    check(H.make([(100, [120, 100])], 2, 128, 16, dtype, heads, seed=9), scale=scale)


def test_long():
    """Runs of many tiles, row tiles that are one run's and that are several's."""
    _say("shared: long")
    check(H.make([(9000, [9100, 9000, 9300] + [9001] * 8), (64, [80] * 3), (3000, [3500, 3001])], 2, 64, 64, BF16, 16, seed=5))
    check(H.make([(70, [75] * 40)] * 9, 16, 128, 16, FP16, 64, seed=6))


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("dim", [128, 200])
@pytest.mark.parametrize("heads", [8, 32])
def test_bad_pages(dtype, dim, heads):
    """Page numbers outside the pool: their tokens are left out, whatever lies where they point."""
    _say("shared: bad pages %s %d" % (dtype, dim))
    m = H.make([(100, [120, 100, 130]), (64, [64, 70])], 2, dim, 16, dtype, heads, seed=1)
    m.table[0, 2] = m.k.shape[0]
    m.table[3, 0] = -1
    m.table[2, 7] = 1 << 30
    hidden = {(b, t) for b in (0, 1, 2) for t in range(32, 48)} | {(b, t) for b in (3, 4) for t in range(16)}
    hidden |= {(2, t) for t in range(112, 128)}
    check(m, hidden=hidden, want_status=_abi.KV_BAD_PAGE)
    # none of the tokens in common
    m = H.make([(32, [40, 32, 33])], 2, dim, 16, dtype, heads, seed=2)
    m.table[0, :2] = -1
    check(m, hidden={(b, t) for b in range(3) for t in range(32)}, want_status=_abi.KV_BAD_PAGE)


def test_ranges_that_decrease():
    _say("shared: ranges that decrease")
    m = H.make([(100, [120, 100, 130]), (64, [64, 70])], 2, 128, 16, BF16, 8, seed=1)
    for cu in ([0, 3, 2], [0, 3, 6], [-1, 2, 2], [3, 3, 1 << 30]):
        m.cu = cu
        check(m, want_status=_abi.KV_BAD_ROWS)
    m.cu, m.shared = [0, 3, 5], [-4, 64]
    check(m, want_status=_abi.KV_BAD_LEN)


@pytest.mark.parametrize("length", [64, 2048])
@pytest.mark.parametrize("groups", [2001, 2049, 65535])
@pytest.mark.parametrize("heads", [1, 32])
def test_ranges_that_overlap_many_times(heads, groups, length):
    """Groups that have all sequences over and over, more work than sums of 32 bits hold: reported, and the call ends."""
    _say("shared: %d ranges that overlap, %d heads, %d tokens" % (groups, heads, length))
    batch, page = 2048, 64
    k = torch.zeros(length // page, 1, page, 64, dtype=BF16, device=DEV)
    table = torch.arange(length // page, dtype=torch.int32, device=DEV).repeat(batch, 1)
    cache = S.KVCache(k, torch.ones_like(k), table, torch.full((batch,), length, dtype=torch.int32, device=DEV))
    q = torch.zeros(batch, heads, 64, dtype=BF16, device=DEV)
    cu = torch.tensor([0, batch] * (groups // 2 + 1), dtype=torch.int32, device=DEV)
    assert cu.numel() == groups + 1
    shared = torch.full((groups,), length, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    cache.attend_shared(q, cu, shared, S.KVSharedWorkspace(cache, heads, groups), status=status)
    torch.cuda.synchronize()
    assert int(status) == _abi.KV_BAD_ROWS


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("members", [3, 20])
def test_infinite_values(dtype, members):
    """An infinity in V of a token in common comes out as one, under small weights too; a NaN in K makes its rows NaN."""
    _say("shared: infinities %s" % dtype)
    m = H.make([(100, [120, 100, 130] + [101] * (members - 3))], 2, 128, 16, dtype, 8, seed=1)
    page = int(m.table[0, 3])
    m.v[page, 1, 5, 7] = float("inf")
    m.v[page, 0, 2, 9] = float("-inf")
    check(m)
    # Logits of a spread of more than 126 powers of two: 32 bits hold no weight below 2^-126 of the largest, and 0
    # times the infinity is a NaN.  Every other output is as it was.
    widen(m)
    R.to_gpu(m, S)
    out = m.cache.attend_shared(m.gq, ints(m.cu), ints(m.shared), S.KVSharedWorkspace(m.cache, 8, 1), scale=2.0)
    small = 0
    for b, (o, tol, _, _) in enumerate(H.attend(m, 2.0)):
        k = R.rows(m, b, range(m.lens[b]), m.k).double()
        for h, j, t, column in [(h, 1, 53, 7) for h in range(4, 8)] + [(h, 0, 50, 9) for h in range(4)]:
            x = 2.0 * (k[:, j] @ m.q[b, h].double()) / math.log(2.0)
            if x[t] < x.max() - 125:
                assert not bool(out[b, h, column].isfinite()), (b, h)
                out[b, h, column] = o[h, column].to(dtype)
                small += 1
        close(out[b], o, tol, "out %d" % b)
    assert 0 < small < 8 * members
    m.k[page, 0, 4, 3] = float("nan")
    R.to_gpu(m, S)
    out = m.cache.attend_shared(m.gq, ints(m.cu), ints(m.shared), S.KVSharedWorkspace(m.cache, 8, 1))
    assert bool(out[:, :4].isnan().all()) and not bool(out[:, 4:, :7].isnan().any())


def test_strides_and_places():
    """Queries and outputs with strides of their own, the output in the queries' place, rows behind them left."""
    _say("shared: strides")
    m = H.make([(100, [120, 100, 130])], 2, 64, 16, BF16, 8, seed=1)
    want = check(m)
    ws = S.KVSharedWorkspace(m.cache, 8, 1)
    q = torch.zeros(8, 4, 80, dtype=BF16, device=DEV).transpose(0, 1)[:3, :, :64]
    q.copy_(m.gq)
    out = torch.full((4, 9, 72), 5.0, dtype=BF16, device=DEV)
    assert m.cache.attend_shared(q, ints(m.cu), ints(m.shared), ws, out=out[:3, :8, :64]).data_ptr() == out.data_ptr()
    assert torch.equal(out[:3, :8, :64], want)
    assert bool((out[3] == 5).all()) and bool((out[:, 8] == 5).all()) and bool((out[..., 64:] == 5).all())
    m.cache.attend_shared(m.gq, ints(m.cu), ints(m.shared), ws, out=m.gq)
    assert torch.equal(m.gq, want)


@pytest.mark.parametrize("many", [False, True])
def test_far_pages(many):
    """Offsets beyond 2^32 elements."""
    _say("shared: far pages")
    m = H.make([(100, [120, 100] * 6)], 1, 128, 16, BF16, 4, seed=2)
    if many:
        widen(m)
    R.to_gpu(m, S)
    ws = S.KVSharedWorkspace(m.cache, 4, 1)
    want = m.cache.attend_shared(m.gq, ints(m.cu), ints(m.shared), ws)
    pages, far = m.k.shape[0], (1 << 32) // (16 * 128) + 11
    k, v = (torch.empty(far + pages, 1, 16, 128, dtype=BF16, device=DEV) for _ in range(2))
    k[far:], v[far:] = m.gk, m.gv
    cache = S.KVCache(k, v, torch.where(m.gtable >= 0, m.gtable + far, -1), m.glens)
    assert torch.equal(cache.attend_shared(m.gq, ints(m.cu), ints(m.shared), ws), want)


class Step:
    def __init__(self, seed, groups):
        self.m = H.make(groups, 2, 64, 16, BF16, 8, seed=seed)
        widen(self.m)
        R.to_gpu(self.m, S)
        self.ws = S.KVSharedWorkspace(self.m.cache, 8, len(groups))
        self.cu, self.shared = ints(self.m.cu), ints(self.m.shared)
        self.out, self.lse = torch.zeros_like(self.m.gq), torch.zeros(len(self.m.lens), 8, device=DEV)

    def fill(self, seed):
        g = torch.Generator().manual_seed(seed)
        self.m.gq.copy_(torch.randn(self.m.gq.shape, generator=g))
        self.out.zero_()
        self.lse.zero_()

    def run(self, stream=None):
        self.m.cache.attend_shared(self.m.gq, self.cu, self.shared, self.ws, out=self.out, lse=self.lse, stream=stream)

    def results(self):
        return [self.out.clone(), self.lse.clone()]


def same(got, want, what):
    for x, y in zip(got, want):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), what


def test_streams_and_graphs():
    _say("shared: two streams, two graphs")
    steps = [Step(1, [(300, [310, 300, 333]), (40, [50, 41])]), Step(2, [(1000, [1100] * 30)])]
    streams = [torch.cuda.Stream() for _ in steps]
    graphs = []
    for s in steps:
        s.fill(0)
        s.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    for rep in range(5):
        want = []
        for i, s in enumerate(steps):
            s.fill(10 * rep + i)
            s.run()
            want.append(s.results())
            s.fill(10 * rep + i)
        torch.cuda.synchronize()
        for i, s in enumerate(steps):
            s.run(streams[i])
        torch.cuda.synchronize()
        for i, s in enumerate(steps):
            same(s.results(), want[i], ("stream", rep))
            s.fill(10 * rep + i)
        torch.cuda.synchronize()
        for i, g in enumerate(graphs):
            with torch.cuda.stream(streams[i]):
                g.replay()
        torch.cuda.synchronize()
        for i, s in enumerate(steps):
            same(s.results(), want[i], ("graph", rep))
