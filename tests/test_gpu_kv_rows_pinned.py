"""Rows in pinned host memory, into the cache and out of it."""
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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim,kv_heads,page,layout", [(128, 8, 16, "nhd"), (64, 3, 7, "hnd"), (200, 2, 24, "nhd")])
def test_append_and_gather_of_pinned_rows(dim, kv_heads, page, layout, dtype):
    """A part of each sequence, rows as slices of pinned ones; what lies around
    them stays."""
    _say("pinned rows dim=%d heads=%d page=%d %s" % (dim, kv_heads, page, layout))
    lens = [0, 1, 2 * page + 1, 77, 1500]
    counts = [n - n // 3 for n in lens]
    m = R.to_gpu(R.make(lens, kv_heads, dim, page, dtype, layout=layout, seed=dim), S)
    total = sum(counts)
    cu = torch.tensor([sum(counts[:b]) for b in range(len(lens) + 1)], dtype=torch.int32, device=DEV)
    new = torch.randn(total + 2, 2 * kv_heads, dim, generator=torch.Generator().manual_seed(1)).to(dtype).pin_memory()
    back = torch.full((total + 2, 2 * kv_heads, dim), 2.5, dtype=dtype).pin_memory()
    k, v = new[:, :kv_heads], new[:, kv_heads:]
    want_k, want_v = m.k.clone(), m.v.clone()
    at = 0
    for b, n in enumerate(lens):
        pos = torch.arange(n - counts[b], n)
        for rows, want in ((k, want_k), (v, want_v)):
            want[m.table[b].long()[pos // page], :, pos % page] = rows[at:at + counts[b]]
        at += counts[b]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.cache.append(k, v, cu, status=status)
    m.cache.gather(back[:, :kv_heads], back[:, kv_heads:], cu, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    assert torch.equal(bits(m.gk.cpu()), bits(want_k)) and torch.equal(bits(m.gv.cpu()), bits(want_v))
    assert torch.equal(bits(back[:total]), bits(new[:total])) and bool((back[total:] == 2.5).all())
