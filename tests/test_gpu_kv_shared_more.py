"""More of the attention over sequences that begin alike: as many shares of one
query head as there are runs."""
import pytest
import torch

import kv_shared_reference as H
from test_gpu_kv_shared import check_one, widen
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
