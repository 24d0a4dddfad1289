"""The key-value cache library on a machine without a GPU: exported symbols,
struct mirrors, workspace sizes and the refusals of every entry point.  No
device work is launched here."""
import ctypes
import os
import re

import pytest
import torch

import lossless_bf16_tensor_splitzip_amd as S
from lossless_bf16_tensor_splitzip_amd import _abi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_declared_symbol_is_exported():
    text = open(os.path.join(ROOT, "include", "splitzip_kv.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(splitzip_kv_\w+)\s*\(", text)))
    assert names == sorted(_abi.KV_SIGNATURES)
    for name in names:
        assert hasattr(_abi.kv_lib(), name), name


def test_structs_match_the_header():
    sizes = (ctypes.c_size_t * 4)()
    _abi.kv_lib().splitzip_kv_struct_sizes(sizes)
    assert list(sizes) == [ctypes.sizeof(t) for t in _abi.KV_STRUCTS] == [120, 72, 128, 72]


def cache(**over):
    a = dict(k=0x10000, v=0x20000, k_stride0=8 * 16 * 64, k_stride1=16 * 64, k_stride2=64, v_stride0=8 * 16 * 64,
             v_stride1=16 * 64, v_stride2=64, table=0x3000, table_stride=4, lens=0x4000, num_pages=10, page_size=16,
             kv_heads=8, head_dim=64, batch=2, max_pages=4, dtype=0, reserved=0)
    a.update(over)
    return _abi.KVCacheArgs(**a)


def rows(**over):
    a = dict(k=0x10000, v=0x20000, k_stride0=512, k_stride1=64, v_stride0=512, v_stride1=64, rows=5, cu=0x5000,
             start=None)
    a.update(over)
    return _abi.KVRows(**a)


def query(**over):
    a = dict(q=0x10000, q_stride0=1024, q_stride1=64, out=0x20000, out_stride0=1024, out_stride1=64, heads=16,
             window=_abi.KV_ALL, sinks=0, scale=0.125)
    a.update(over)
    return _abi.KVQuery(**a)


def budget(**over):
    a = dict(mass=0x10000, mass_out=0x10000, mass_stride0=512, mass_stride1=64, mass_out_stride0=512,
             mass_out_stride1=64, kept=0x9000, budget=32, sinks=4, recent=8, mass_len=64)
    a.update(over)
    return _abi.KVBudget(**a)


BAD_CACHES = [
    dict(k=0), dict(v=None), dict(k=0x10008), dict(v=0x20002), dict(head_dim=0), dict(head_dim=4), dict(head_dim=65),
    dict(head_dim=264), dict(kv_heads=0), dict(kv_heads=4097), dict(page_size=0), dict(page_size=65537),
    dict(num_pages=0), dict(num_pages=1 << 31), dict(batch=65536), dict(dtype=2), dict(k_stride0=4),
    dict(k_stride2=65), dict(v_stride1=12), dict(k_stride0=1 << 37), dict(v_stride0=(1 << 64) - 8), dict(lens=0),
    dict(lens=0x4002), dict(table=0), dict(table=0x3002), dict(table_stride=3), dict(max_pages=1 << 27),
    dict(max_pages=0xFFFFFFFF, page_size=65536, table_stride=1 << 32)]


@pytest.mark.parametrize("over", BAD_CACHES, ids=str)
def test_bad_caches_are_refused(over):
    c = cache(**over)
    assert _abi.splitzip_kv_append(c, rows(), 0, 0) == _abi.ERR_INVALID
    assert _abi.splitzip_kv_gather(c, rows(), 0, 0) == _abi.ERR_INVALID
    assert _abi.splitzip_kv_attend(c, query(), 0x8000, 1 << 40, 0, 0) == _abi.ERR_INVALID
    assert _abi.splitzip_kv_evict(c, cache(), budget(), 0, 0) == _abi.ERR_INVALID
    assert _abi.splitzip_kv_evict(cache(), c, budget(), 0, 0) == _abi.ERR_INVALID


@pytest.mark.parametrize("over", [dict(k=0), dict(v=0x20008), dict(k_stride0=9), dict(v_stride1=4), dict(cu=0),
                                  dict(cu=0x5001), dict(start=0x6002), dict(rows=0x80000000),
                                  dict(k_stride0=1 << 39)], ids=str)
def test_bad_rows_are_refused(over):
    for fn in (_abi.splitzip_kv_append, _abi.splitzip_kv_gather):
        assert fn(cache(), rows(**over), 0, 0) == _abi.ERR_INVALID


@pytest.mark.parametrize("over", [dict(q=0), dict(q=0x10008), dict(out=0), dict(out=0x20004), dict(q_stride0=4),
                                  dict(out_stride1=1 << 41), dict(heads=0), dict(heads=12), dict(heads=65536),
                                  dict(lse=0x7001), dict(mass=0x7000), dict(mass_out=0x7002),
                                  dict(scale=float("nan")), dict(scale=float("inf")),
                                  dict(scale=3e38)], ids=str)
def test_bad_queries_are_refused(over):
    assert _abi.splitzip_kv_attend(cache(), query(**over), 0x8000, 1 << 40, 0, 0) == _abi.ERR_INVALID


def test_workspace_and_status_are_checked():
    need = _abi.splitzip_kv_attend_workspace_size(cache(), 16, 0)
    assert need > 0
    assert _abi.splitzip_kv_attend(cache(), query(), 0x8000, need - 1, 0, 0) == _abi.ERR_WORKSPACE
    assert _abi.splitzip_kv_attend(cache(), query(), 0, need, 0, 0) == _abi.ERR_INVALID
    assert _abi.splitzip_kv_attend(cache(), query(), 0x8008, need, 0, 0) == _abi.ERR_INVALID
    assert _abi.splitzip_kv_attend(cache(), query(), 0x8000, need, 2, 0) == _abi.ERR_INVALID
    assert _abi.splitzip_kv_append(cache(), rows(), 1, 0) == _abi.ERR_INVALID
    assert _abi.splitzip_kv_evict(cache(), cache(), budget(), 6, 0) == _abi.ERR_INVALID
    with_mass = _abi.splitzip_kv_attend_workspace_size(cache(), 16, 64)
    assert with_mass >= need
    q = query(mass_out=0x7000, mass_len=64)
    assert _abi.splitzip_kv_attend(cache(), q, 0x8000, with_mass - 1, 0, 0) == _abi.ERR_WORKSPACE
    # shapes without a size
    for over, heads in ((dict(), 0), (dict(), 12), (dict(head_dim=7), 16), (dict(dtype=3), 16)):
        assert _abi.splitzip_kv_attend_workspace_size(cache(**over), heads, 0) == 0


@pytest.mark.parametrize("over", [dict(mass=0), dict(mass=0x10002), dict(mass_out=0x10001), dict(kept=0),
                                  dict(kept=0x9002), dict(budget=0), dict(budget=1 << 31), dict(sinks=33),
                                  dict(sinks=20, recent=13), dict(recent=0xFFFFFFFF), dict(mass_stride0=1 << 41)],
                         ids=str)
def test_bad_budgets_are_refused(over):
    assert _abi.splitzip_kv_evict(cache(), cache(), budget(**over), 0, 0) == _abi.ERR_INVALID


@pytest.mark.parametrize("over", [dict(k=0x90000), dict(table=0x93000), dict(lens=0x94000), dict(page_size=8),
                                  dict(batch=1), dict(kv_heads=4), dict(head_dim=128), dict(dtype=1),
                                  dict(k_stride2=72),
                                  dict(k=0x90000, v=0xA0000, table=0x93000, lens=0x94000, max_pages=1)], ids=str)
def test_bad_destinations_are_refused(over):
    """A destination that shares something with the cache without being it,
    differs in shape, or is too small for the budget."""
    assert _abi.splitzip_kv_evict(cache(), cache(**over), budget(), 0, 0) == _abi.ERR_INVALID


def test_empty_calls_launch_nothing():
    empty = cache(batch=0, table=None, lens=None)
    assert _abi.splitzip_kv_append(empty, rows(), 0, 0) == _abi.OK
    assert _abi.splitzip_kv_gather(cache(), rows(rows=0, k=None, v=None), 0, 0) == _abi.OK
    assert _abi.splitzip_kv_attend(empty, query(q=None, out=None), 0, 1 << 30, 0, 0) == _abi.OK
    assert _abi.splitzip_kv_evict(empty, empty, budget(), 0, 0) == _abi.OK


def test_binding_refuses_host_tensors():
    pool = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        S.KVCache(pool, pool.clone(), table, lens)
    with pytest.raises(ValueError):
        S.KVCache(pool.float(), pool.float(), table, lens)
