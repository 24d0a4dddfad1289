"""Lengths that no table can hold, where a sequence leaves or arrives."""
import types

import pytest
import torch

import lossless_bf16_tensor_splitzip_amd as S
import kv_reference as R


def _say(msg):
    print("[kv persist] " + msg, flush=True)


@pytest.mark.parametrize("n", [-1, -2 ** 31, 65, 2 ** 31 - 1])
def test_a_length_outside_its_table_does_not_leave(n):
    """Named for what it is, before anything is read."""
    cache = types.SimpleNamespace(batch=2, lens=torch.tensor([64, n], dtype=torch.int32), max_pages=4, page_size=16)
    with pytest.raises(ValueError, match="a length of %d, .* 0 to 64 tokens" % n):
        S.persist.pack_sequence("x", cache, 1, None)


def test_what_a_status_says():
    for bits, text in ((1, "pages outside the pool"), (3, "pages outside the pool"), (4, "no place"), (2, "no place")):
        with pytest.raises(ValueError, match=text):
            S.persist._check_placed(torch.tensor([bits], dtype=torch.int32), 0)
    S.persist._check_placed(torch.zeros(1, dtype=torch.int32), 0)


@pytest.mark.gpu
@pytest.mark.parametrize("old", [-1, 1 << 30, -2 ** 31, 4, 0])
def test_a_sequence_arrives_whatever_its_length_was(old):
    _say("arrives over a length of %d" % old)
    n = 333
    m = R.to_gpu(R.make([40, n, 7], 4, 128, 16, torch.bfloat16, seed=n), S)
    packed = S.persist.pack_sequence("x", m.cache, 1, S.Workspace(n * 4 * 128, "cuda:0"))
    want = m.gk.clone(), m.gv.clone()
    for pool in (m.gk, m.gv):
        pool[m.gtable[1].long()] = 3.0
    m.glens[1] = old
    assert S.persist.unpack_sequence(packed, m.cache, 1) == n
    assert m.glens.tolist() == [40, n, 7]
    for pool, old_pool in ((m.gk, want[0]), (m.gv, want[1])):
        got, kept = (R.rows(m, 1, torch.arange(n), p.cpu()).contiguous().view(torch.int16) for p in (pool, old_pool))
        assert torch.equal(got, kept)


@pytest.mark.gpu
@pytest.mark.parametrize("fn", ["append", "gather"])
def test_rows_with_first_positions_do_not_look_at_lengths(fn):
    _say("%s with first positions" % fn)
    m = R.to_gpu(R.make([40, 20], 2, 64, 16, torch.bfloat16, seed=3, fill=1.0), S)
    k, v = (torch.randn(12, 2, 64, device="cuda:0").to(torch.bfloat16) for _ in range(2))
    cu = torch.tensor([0, 5, 12], dtype=torch.int32, device="cuda:0")
    start = torch.tensor([30, 3], dtype=torch.int32, device="cuda:0")
    status = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    m.glens.copy_(torch.tensor([-5, 1 << 30], dtype=torch.int32))
    getattr(m.cache, fn)(k, v, cu, start=start, status=status)
    assert int(status) == 0
    for b, (first, count, row) in enumerate(((30, 5, 0), (3, 7, 5))):
        pos = torch.arange(first, first + count)
        for rows, pool in ((k, m.gk), (v, m.gv)):
            assert torch.equal(rows[row:row + count].cpu(), R.rows(m, b, pos, pool.cpu()))
    # without them they are judged
    getattr(m.cache, fn)(k, v, cu, status=status)
    assert int(status) & 2
