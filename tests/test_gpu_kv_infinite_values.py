"""Infinities in V under small weights: infinite in their columns, as the
formula has them, wherever the token lies before or behind the largest."""
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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim,heads,width", [(64, 1, None), (128, 20, None), (72, 3, None), (256, 2, None),
                                             (128, 4, 600), (64, 40, 600)])
@pytest.mark.parametrize("depth", [10, 27, 28, 30, 45, 60, 80])
def test_infinite_v_under_a_small_weight(dtype, dim, heads, width, depth):
    """The weight is e^-depth of the largest (e^-87 is 2^-126, the smallest
    normal number of 32 bits).  Tokens 30 (in the largest's tile), 3 (before
    it) and 600 (tiles behind it) hold the infinities, in columns of their own."""
    _say("infinite V %d nats down dim=%d heads=%d wide=%s %s" % (depth, dim, heads, width, dtype))
    n, top = 700, 20
    m = R.make([n], 1, dim, 16, dtype, heads=heads, seed=depth, width=width)
    t = torch.arange(n)
    where, slot = m.table[0].long()[t // 16], t % 16
    m.q[:] = 0.0
    m.q[:, :, 0] = 1.0
    m.k[where, 0, slot, 0] = torch.where(t == top, 0.0, -float(depth)).to(dtype)
    for tok in (3, 30, 600):
        m.v[where[tok], 0, slot[tok]] = 0.0
    want = R.attend(m, scale=1.0)[0]
    cols = torch.zeros(dim, dtype=torch.float64)
    for tok, col, x in ((3, 1, math.inf), (30, dim - 1, -math.inf), (600, dim // 2, math.inf)):
        m.v[where[tok], 0, slot[tok], col] = x
        cols[col] = x
    R.to_gpu(m, S)
    out = m.cache.attend(m.gq, S.KVWorkspace(m.cache, heads), scale=1.0)[0].double().cpu()
    hit = cols != 0
    assert torch.equal(out[:, hit], cols[hit].expand(heads, -1))
    assert bool(((out - want[0]).abs() <= want[1])[:, ~hit].all())
