"""Rows into and out of a paged cache: bit-exact copies."""
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


def cu_of(counts):
    cu = [0]
    for n in counts:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dim,kv_heads,page,layout,dtype", [
    (128, 8, 16, "nhd", torch.bfloat16), (128, 8, 16, "hnd", torch.bfloat16), (64, 3, 7, "nhd", torch.float16),
    (8, 1, 1, "hnd", torch.bfloat16), (256, 2, 100, "hnd", torch.float16), (200, 5, 24, "nhd", torch.bfloat16),
    (256, 40, 8, "hnd", torch.bfloat16)])
@pytest.mark.parametrize("case", ["all", "one", "part", "start"])
def test_append_and_gather(dim, kv_heads, page, layout, dtype, case):
    _say("rows dim=%d heads=%d page=%d %s %s" % (dim, kv_heads, page, layout, case))
    lens = [0, 1, page, 2 * page + 1, 77, 300]
    counts = {"all": lens, "one": [min(n, 1) for n in lens], "part": [n // 2 for n in lens],
              "start": [n // 3 for n in lens]}[case]
    start = torch.tensor([n // 2 for n in lens], dtype=torch.int32, device=DEV) if case == "start" else None
    m = R.to_gpu(R.make(lens, kv_heads, dim, page, dtype, layout=layout, seed=dim), S)
    total, extra = sum(counts), 3
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    # gather: rows with the head dimension outermost, as the encoder takes them
    k, v = (torch.full((kv_heads, total + extra, dim), 2.5, dtype=dtype, device=DEV).transpose(0, 1) for _ in range(2))
    m.cache.gather(k, v, cu_of(counts), start=start, status=status)
    want_k, want_v = m.k.clone(), m.v.clone()
    new_k, new_v = (torch.randn(total + extra, kv_heads, dim, device=DEV).to(dtype) for _ in range(2))
    at = 0
    for b, n in enumerate(lens):
        first = n - counts[b] if start is None else n // 2
        pos = torch.arange(first, first + counts[b])
        for got, pool, new, want in ((k, m.k, new_k, want_k), (v, m.v, new_v, want_v)):
            assert torch.equal(bits(got[at:at + counts[b]].cpu()), bits(R.rows(m, b, pos, pool))), b
            want[m.table[b].long()[pos // page], :, pos % page] = new[at:at + counts[b]].cpu()
        at += counts[b]
    assert bool((k[total:] == 2.5).all()) and bool((v[total:] == 2.5).all())
    m.cache.append(new_k, new_v, cu_of(counts), start=start, status=status)
    assert torch.equal(bits(m.gk.cpu()), bits(want_k)) and torch.equal(bits(m.gv.cpu()), bits(want_v))
    assert int(status) == 0


def test_long_prompt_and_strided_rows():
    """A prompt of 20,000 tokens; K and V as slices of one projection's rows;
    rows in pinned host memory."""
    n = 20000
    m = R.to_gpu(R.make([n], 2, 64, 16, torch.bfloat16, seed=2), S)
    qkv = torch.randn(n, 8, 64, device=DEV).to(torch.bfloat16)
    m.cache.append(qkv[:, 4:6], qkv[:, 6:8], cu_of([n]))
    k, v = (torch.empty(n, 2, 64, dtype=torch.bfloat16).pin_memory() for _ in range(2))
    m.cache.gather(k, v, cu_of([n]))
    torch.cuda.synchronize()
    assert torch.equal(bits(k), bits(qkv[:, 4:6].cpu())) and torch.equal(bits(v), bits(qkv[:, 6:8].cpu()))


def test_bad_places_are_left_out():
    m = R.to_gpu(R.make([40, 20], 1, 64, 16, torch.bfloat16, seed=3, fill=1.0), S)
    before = m.gk.clone(), m.gv.clone()
    k, v = (torch.randn(60, 1, 64, device=DEV).to(torch.bfloat16) for _ in range(2))

    def call(want, cu, start=None, untouched=True):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        if start is not None:
            start = torch.tensor(start, dtype=torch.int32, device=DEV)
        m.cache.append(k, v, torch.tensor(cu, dtype=torch.int32, device=DEV), start=start, status=status)
        assert int(status) == want
        if untouched:
            assert torch.equal(m.gk, before[0]) and torch.equal(m.gv, before[1])

    call(4, [0, 61, 61], [0, 0])               # a range past the rows
    call(4, [0, 1, 1], [48, 0])                # behind the table's end
    call(4, [0, 2, 2], [-2, 0])
    call(0, [0, 0, 0])
    call(0, [60, 60, 60])
    m.gtable[0, 0] = m.gk.shape[0]
    call(1, [0, 16, 16], [0, 0])
    m.gtable[0, 0] = -1
    call(1, [0, 16, 16], [0, 0])


def test_rows_below_zero_do_not_stop_the_others():
    m = R.to_gpu(R.make([10, 20], 1, 64, 16, torch.bfloat16, seed=3, fill=1.0), S)
    k, v = (torch.randn(32, 1, 64, device=DEV).to(torch.bfloat16) for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.cache.append(k, v, cu_of([12, 20]), status=status)
    got = m.gk.cpu()
    assert int(status) == 4
    for b, first, n, row in ((0, 0, 10, 2), (1, 0, 20, 12)):
        pos = torch.arange(first, n)
        assert torch.equal(bits(R.rows(m, b, pos, got)), bits(k[row:row + n].cpu()))


def test_graph_replays_of_a_step():
    """The step's append inside a graph: the lengths and tokens change between
    the replays, the batch is padded with sequences of no tokens."""
    m = R.to_gpu(R.make([5, 16, 0, 40], 2, 64, 16, torch.bfloat16, seed=5, width=4, slack=9), S)
    free = [p for p in range(m.k.shape[0]) if p not in m.table.tolist()[0] + m.table.tolist()[1] + m.table.tolist()[3]]
    m.gtable[1, 1] = m.table[1, 1] = free[0]
    k, v = (torch.empty(4, 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    cu = torch.tensor([0, 1, 2, 2, 3], dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.cache.append(k, v, cu)
    want = m.gk.cpu()
    for rep in range(6):
        m.glens.add_(torch.tensor([1, 1, 0, 1], dtype=torch.int32, device=DEV))
        k.copy_(torch.randn(4, 2, 64, device=DEV))
        g.replay()
        torch.cuda.synchronize()
        for row, b in enumerate((0, 1, 3)):
            t = int(m.glens[b]) - 1
            want[m.table[b, t // 16].long(), :, t % 16] = k[row].cpu()
        assert torch.equal(bits(m.gk.cpu()), bits(want)), rep
