"""Attention asked for a mass of no tokens: no weight has a place, and
sequences that have tokens are reported as too long for it."""
import pytest
import torch

import lossless_bf16_tensor_splitzip_amd as S
import kv_reference as R
from test_gpu_parity import DEV, _say

pytestmark = pytest.mark.gpu


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("lens,width,want", [([40, 0, 3], None, 2), ([0, 0], None, 0), ([900, 0, 1], 600, 2), ([0], 600, 0)])
def test_a_mass_of_no_tokens(lens, width, want):
    _say("a mass of no tokens, lengths %s" % lens)
    m = R.to_gpu(R.make(lens, 2, 64, 16, torch.bfloat16, heads=4, seed=3, width=width), S)
    plain = m.cache.attend(m.gq, S.KVWorkspace(m.cache, 4))
    ws = S.KVWorkspace(m.cache, 4, mass=True)
    for names in (("mass",), ("mass_out",), ("mass", "mass_out")):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        masses = {name: torch.zeros(len(lens), 2, 0, device=DEV) for name in names}
        out = m.cache.attend(m.gq, ws, status=status, **masses)
        assert int(status) == want
        assert torch.equal(out.view(torch.int16), plain.view(torch.int16)) and m.glens.tolist() == lens
