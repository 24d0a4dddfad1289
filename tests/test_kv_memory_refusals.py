"""kv_memory_checks without a GPU: host tensors that say they are on one, and
the real library, in which a call that is accepted gets as far as the launch."""
import pytest
import torch

import lossless_bf16_tensor_splitzip_amd as S
from lossless_bf16_tensor_splitzip_amd import _abi, kv
import kv_memory_checks
from test_kv_refusals import SaysGpu


@pytest.mark.skipif(torch.cuda.is_available(), reason="accepted calls would launch on host memory")
@pytest.mark.parametrize("part", kv_memory_checks.PARTS)
def test_refusals(part, monkeypatch):
    monkeypatch.setattr(kv, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(S.KVWorkspace, "_buffer", lambda self, nbytes, device: put(torch.empty(nbytes, dtype=torch.uint8)))

    def put(t):
        return t.as_subclass(SaysGpu)

    def to_gpu(m):
        m.gk, m.gv, m.gtable = put(m.k.clone()), put(m.v.clone()), put(m.table)
        m.glens = put(torch.tensor(m.lens, dtype=torch.int32))
        m.cache = S.KVCache(m.gk, m.gv, m.gtable, m.glens)
        if hasattr(m, "q"):
            m.gq = put(m.q)
        return m

    def runs(fn, *args, **kw):
        with pytest.raises(S.SplitZipError) as e:
            fn(*args, **kw)
        assert e.value.status == _abi.ERR_HIP

    getattr(kv_memory_checks, part)(lambda make, *a, **kw: put(make(*a, **kw)), to_gpu, runs)
