"""The refusals of the page operators and of the attention over sequences that
begin alike, on the GPU."""
import pytest
import torch

import lossless_bf16_tensor_splitzip_amd as S
import kv_pages_checks
import kv_reference as R
from test_gpu_parity import DEV

pytestmark = pytest.mark.gpu


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("part", kv_pages_checks.PARTS)
def test_refusals(part):
    def runs(fn, *args, **kw):
        fn(*args, **kw)
        torch.cuda.synchronize()

    made = S.KVPages._buffer
    try:
        S.KVPages._buffer = lambda self, nbytes, device: torch.zeros(nbytes, dtype=torch.uint8, device=device)
        getattr(kv_pages_checks, part)(lambda make, *a, **kw: make(*a, device=DEV, **kw), lambda m: R.to_gpu(m, S), runs)
    finally:
        S.KVPages._buffer = made
