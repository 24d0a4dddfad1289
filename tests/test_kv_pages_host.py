"""The page operators and the attention over sequences that begin alike at the
C ABI on a machine without a GPU: struct mirrors, sizes and refusals.  No device
work is launched here."""
import ctypes

import pytest

from lossless_bf16_tensor_splitzip_amd import _abi
from test_kv_host import BAD_CACHES, cache, query


def pages(layers=1, state=0x100000, state_bytes=None, c=None, k=None, v=None, **over):
    c = cache(**over) if c is None else c
    ks = (ctypes.c_void_p * max(layers, 1))(*([0x1000000 * (i + 1) for i in range(layers)] if k is None else k))
    vs = (ctypes.c_void_p * max(layers, 1))(*([0x1000000 * (i + 1) + 0x800000 for i in range(layers)] if v is None else v))
    if state_bytes is None:
        state_bytes = 1 << 40
    p = _abi.KVPagesArgs(ctypes.addressof(c), ctypes.addressof(ks), ctypes.addressof(vs), layers, 0, state, state_bytes)
    p.keep = c, ks, vs
    return p


def calls(p, other=None):
    other = pages() if other is None else other
    yield _abi.splitzip_kv_pages_count(p, 0, 0)
    yield _abi.splitzip_kv_pages_fork(p, 0x5000, 0, 0)
    yield _abi.splitzip_kv_pages_resize(p, 0x5000, 0, 0)
    yield _abi.splitzip_kv_pages_compact(p, 0, 0, 0, 0)


def copies(p, other):
    yield _abi.splitzip_kv_pages_copy(p, other, 0x5000, 0x6000, 3, 0, 0)
    yield _abi.splitzip_kv_pages_copy(other, p, 0x5000, 0x6000, 3, 0, 0)


def groups(**over):
    a = dict(cu=0x5000, shared=0x6000, groups=1, reserved=0)
    a.update(over)
    return _abi.KVGroups(**a)


def test_structs_match_the_header():
    assert _abi.splitzip_kv_pages_struct_size() == ctypes.sizeof(_abi.KVPagesArgs) == 48
    assert _abi.splitzip_kv_groups_struct_size() == ctypes.sizeof(_abi.KVGroups) == 24


@pytest.mark.parametrize("over", [o for o in BAD_CACHES if not {"k", "v"} & set(o)], ids=str)
def test_bad_caches_are_refused(over):
    bad = pages(**over)
    assert set(calls(bad)) == {_abi.ERR_INVALID}
    if not {"lens", "table", "table_stride", "batch"} & set(over):        # which a copy does not look at
        assert set(copies(bad, pages())) == {_abi.ERR_INVALID}
    assert _abi.splitzip_kv_attend_shared(cache(**over), query(), groups(), 0x8000, 1 << 40, 0, 0) == _abi.ERR_INVALID


@pytest.mark.parametrize("over", [dict(layers=0), dict(layers=1025), dict(k=[0]), dict(v=[0x1000008]), dict(num_pages=(1 << 24) + 1),
                                  dict(page_size=65536, kv_heads=4096, head_dim=256)], ids=str)
def test_bad_pools_are_refused(over):
    bad = pages(**over)
    assert set(calls(bad)) == {_abi.ERR_INVALID}
    assert set(copies(bad, pages())) == {_abi.ERR_INVALID}


def test_state_and_arguments_are_checked():
    need = _abi.splitzip_kv_pages_state_size(cache())
    assert need >= 6 * 4 * 10
    assert set(calls(pages(state_bytes=need - 1))) == {_abi.ERR_WORKSPACE}
    for state in (0, 0x100008):
        assert set(calls(pages(state=state))) == {_abi.ERR_INVALID}
    good = pages()
    for fn in (_abi.splitzip_kv_pages_fork, _abi.splitzip_kv_pages_resize):
        assert fn(good, 0, 0, 0) == _abi.ERR_INVALID
        assert fn(good, 0x5002, 0, 0) == _abi.ERR_INVALID
        assert fn(good, 0x5000, 2, 0) == _abi.ERR_INVALID
    assert _abi.splitzip_kv_pages_count(good, 2, 0) == _abi.ERR_INVALID
    for moved, used in ((0x5001, 0), (0, 0x5002)):
        assert _abi.splitzip_kv_pages_compact(good, moved, used, 0, 0) == _abi.ERR_INVALID
    # a table of 2^31 entries
    assert set(calls(pages(batch=65535, max_pages=65535, table_stride=65535, page_size=1))) == {_abi.ERR_INVALID}
    for over in (dict(num_pages=0), dict(num_pages=(1 << 24) + 1), dict(batch=65536), dict(head_dim=7)):
        assert _abi.splitzip_kv_pages_state_size(cache(**over)) == 0
    for b in (0, 1, 65535):
        sizes = [_abi.splitzip_kv_pages_state_size(cache(num_pages=n, batch=b)) for n in (1, 256, 257, 1 << 24)]
        assert sorted(sizes) == sizes and all(n >= 6 * 4 * p for n, p in zip(sizes, (1, 256, 257, 1 << 24)))


@pytest.mark.parametrize("over", [dict(page_size=8), dict(kv_heads=4), dict(head_dim=128), dict(dtype=1), dict(layers=2)], ids=str)
def test_copies_between_pools_that_differ_are_refused(over):
    assert set(copies(pages(), pages(**over))) == {_abi.ERR_INVALID}


def test_bad_copies_are_refused():
    a, b = pages(), pages(k=[0x9000000], v=[0xA000000])
    for src, dst, n, status in ((0, 0x6000, 3, 0), (0x5000, 0, 3, 0), (0x5001, 0x6000, 3, 0), (0x5000, 0x6002, 3, 0),
                                (0x5000, 0x6000, 1 << 31, 0), (0x5000, 0x6000, 3, 1)):
        assert _abi.splitzip_kv_pages_copy(a, b, src, dst, n, status, 0) == _abi.ERR_INVALID


def test_empty_calls_launch_nothing():
    empty = pages(batch=0, table=None, lens=None)
    assert _abi.splitzip_kv_pages_fork(empty, 0, 0, 0) == _abi.OK
    assert _abi.splitzip_kv_pages_resize(empty, 0, 0, 0) == _abi.OK
    assert _abi.splitzip_kv_pages_copy(pages(), pages(), 0, 0, 0, 0, 0) == _abi.OK
    none = cache(batch=0, table=None, lens=None)
    assert _abi.splitzip_kv_attend_shared(none, query(q=None, out=None), groups(), 0, 1 << 30, 0, 0) == _abi.OK


@pytest.mark.parametrize("over", [dict(q=0), dict(q=0x10008), dict(out=0), dict(out=0x20004), dict(q_stride0=4),
                                  dict(out_stride1=1 << 41), dict(heads=0), dict(heads=12), dict(heads=65536), dict(lse=0x7001),
                                  dict(mass=0x7000), dict(mass_out=0x7000), dict(window=100), dict(scale=float("nan")),
                                  dict(scale=3e38)], ids=str)
def test_bad_queries_are_refused(over):
    assert _abi.splitzip_kv_attend_shared(cache(), query(**over), groups(), 0x8000, 1 << 40, 0, 0) == _abi.ERR_INVALID


@pytest.mark.parametrize("over", [dict(cu=0), dict(shared=0), dict(cu=0x5002), dict(shared=0x6001), dict(groups=65536)], ids=str)
def test_bad_groups_are_refused(over):
    assert _abi.splitzip_kv_attend_shared(cache(), query(), groups(**over), 0x8000, 1 << 40, 0, 0) == _abi.ERR_INVALID


def test_workspaces_of_the_shared_attention():
    need = _abi.splitzip_kv_shared_workspace_size(cache(), 16, 1)
    assert need > 0
    for n in (0, 1, 7, 65535):                       # one made for more groups serves fewer
        assert _abi.splitzip_kv_shared_workspace_size(cache(), 16, n) == need
    assert _abi.splitzip_kv_attend_shared(cache(), query(), groups(), 0x8000, 64, 0, 0) == _abi.ERR_WORKSPACE
    assert _abi.splitzip_kv_attend_shared(cache(), query(), groups(), 0x8008, need, 0, 0) == _abi.ERR_INVALID
    assert _abi.splitzip_kv_attend_shared(cache(), query(), groups(), 0, need, 0, 0) == _abi.ERR_INVALID
    assert _abi.splitzip_kv_attend_shared(cache(), query(), groups(), 0x8000, need, 2, 0) == _abi.ERR_INVALID
    for over, heads, n in ((dict(), 0, 1), (dict(), 12, 1), (dict(head_dim=7), 16, 1), (dict(), 16, 65536),
                           (dict(max_pages=1 << 26, table_stride=1 << 26, batch=65535), 16, 1),
                           (dict(batch=65535, kv_heads=4096), 65535 // 4096 * 4096, 1)):
        assert _abi.splitzip_kv_shared_workspace_size(cache(**over), heads, n) == 0, over
