"""More of the attention over sequences that begin alike: as many shares of one
query head as there are runs."""
import pytest
import torch

import kv_shared_reference as H
from lossless_bf16_tensor_splitzip_amd import _abi
from test_gpu_kv_shared import check_one, close, widen
from test_gpu_parity import _say

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_every_run_has_a_share():
    """One KV head of one sequence, which all runs have part of; and of a group's tokens in common, in both kernels."""
    _say("shared: all runs' shares of one head")
    check_one(H.make([(0, [100_007])], 1, 64, 64, BF16, 2, seed=1), None, (), 0)
    m = H.make([(131_100, [131_100 + 5 * i for i in range(17)])], 1, 64, 64, FP16, 1, seed=2)
    check_one(m, None, (), 0)
    assert widen(m)
    check_one(m, None, (), 0)


@pytest.mark.parametrize("groups", [2047, 2048, 2049, 65535])
@pytest.mark.parametrize("scale", [0.0, 0.125])
def test_findings_in_many_groups(groups, scale):
    """Ranges that leave the batch or decrease, and fewer than no tokens in common, are reported however many groups there
    are, also where the scale makes no order of logits."""
    _say("shared: findings in %d groups, scale %g" % (groups, scale))
    m = H.make([(100, [120, 100, 130]), (64, [64, 70])], 2, 64, 16, BF16, 4, seed=1)
    m.cu, m.shared = [0, 3, 5] + [5] * (groups - 2), [100, 64] + [0] * (groups - 2)
    check_one(m, scale, (), 0)
    m.shared[-1] = -1
    check_one(m, scale, (), _abi.KV_BAD_LEN)
    m.cu[-2:], m.shared[-1] = [6, 5], 0
    check_one(m, scale, (), _abi.KV_BAD_ROWS)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("dim", [64, 80, 128, 192, 256])
@pytest.mark.parametrize("group", [1, 3, 8, 20])
def test_weights_that_are_not_rounded(dtype, dim, group):
    """Where query rows are few the weights of tokens in common are held like the others': bounds without their rounding."""
    _say("shared: weights in 32 bits, dim=%d group=%d %s" % (dim, group, dtype))
    m = H.make([(500, [520, 500, 533, 700]), (140, [141, 600])], 2, dim, 16, dtype, 2 * group, seed=dim + group, width=45)
    common, m.shared = m.shared, [0, 0]
    want = H.attend(m)
    m.shared = common
    out = check_one(m, None, (), 0)
    for b, (o, tol, _, _) in enumerate(want):
        close(out[b], o, tol, "out %d" % b)
