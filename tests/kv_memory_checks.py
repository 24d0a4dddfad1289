"""More of what the tensor-level calls of the key-value cache refuse: tensors
that meet in memory.  Written like kv_checks, for a run without a GPU and one
with it."""
import torch

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


PARTS = ("tables",)
