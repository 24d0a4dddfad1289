"""Attention where a workgroup's run is several units of 128 tokens long, begins
and ends inside KV heads, and where a KV head has more shares than the join
loads ahead; and kernels that only wide tables or odd head sizes choose."""
import pytest
import torch

import lossless_bf16_tensor_splitzip_amd as S
import kv_reference as R
from test_gpu_kv_attend import check
from test_gpu_parity import _say

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("dim,kv_heads,heads,layout", [(128, 4, 8, "hnd"), (128, 2, 48, "nhd"), (256, 2, 4, "nhd"),
                                                       (256, 1, 24, "hnd"), (64, 5, 10, "nhd"), (80, 4, 4, "hnd")])
def test_runs_of_several_units(dim, kv_heads, heads, layout, dtype):
    """564 units of 128 tokens a KV head over 256 to 768 runs."""
    _say("attend runs of several units dim=%d heads=%d/%d %s" % (dim, heads, kv_heads, dtype))
    lens = [30000, 0, 12345, 20001, 777, 9000, 1]
    m = R.make(lens, kv_heads, dim, 16, dtype, layout=layout, heads=heads, seed=dim + heads)
    check(R.to_gpu(m, S))
    check(m, window=9001, sinks=130)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("dim,heads", [(64, 2), (128, 1), (128, 20), (256, 3), (96, 2)])
def test_one_head_of_many_shares(dim, heads, dtype):
    """One sequence, one KV head: a share for each of its 256 units."""
    _say("attend 256 shares dim=%d heads=%d %s" % (dim, heads, dtype))
    check(R.to_gpu(R.make([32700], 1, dim, 64, dtype, heads=heads, seed=dim), S))


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("dim,group", [(24, 64), (40, 48), (56, 64), (64, 50), (72, 64), (104, 33), (120, 64), (128, 64)])
def test_blocks_of_64_rows_in_wide_tables(dim, group, dtype):
    """Tables for 13120 tokens: 5 sequences of 2 KV heads are 1030 units, from
    where on the 64-row kernels are taken; cut into runs, and whole."""
    _say("attend 64 rows dim=%d group=%d %s" % (dim, group, dtype))
    m = R.make([40, 0, 1333, 129, 1], 2, dim, 16, dtype, heads=2 * group, seed=dim, width=820)
    check(R.to_gpu(m, S))
    check(m, window=100, sinks=3)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("dim,group", [(136, 4), (168, 1), (184, 16), (192, 5), (216, 7), (248, 16)])
def test_one_block_of_wide_odd_dims(dim, group, dtype):
    _say("attend one block of rows dim=%d group=%d %s" % (dim, group, dtype))
    for width in (None, 500):
        check(R.to_gpu(R.make([40, 0, 333, 129, 1], 2, dim, 16, dtype, heads=2 * group, seed=dim, width=width), S))


@pytest.mark.parametrize("dim,kv_heads,heads", [(128, 4, 16), (256, 2, 24)])
def test_repeats_of_long_runs_are_bit_equal(dim, kv_heads, heads):
    """The same bits from every pass, others between them and none waited for."""
    ms = [R.to_gpu(R.make([30000, 777, 0, 20001, 9000], kv_heads, dim, 16, BF16, heads=heads, seed=i), S) for i in range(2)]
    ws = [S.KVWorkspace(m.cache, heads, mass=True) for m in ms]

    def run(i):
        mass = torch.zeros(5, kv_heads, 30000, device="cuda:0")
        return ms[i].cache.attend(ms[i].gq, ws[i], mass=mass), mass

    first = [run(0), run(1)]
    for rep in range(20):
        later = [run(0), run(1), run(0)]
        for (o, mass), (o0, mass0) in zip(later, first + first[:1]):
            assert torch.equal(o.view(torch.int16), o0.view(torch.int16)) and torch.equal(mass, mass0), rep
