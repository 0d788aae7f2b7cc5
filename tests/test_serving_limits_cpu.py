"""The sizes that the cache calls accept, and the next ones, which they refuse (no pointer is followed)."""
import ctypes

import pytest

import precision_attention_nvfp4_b200 as fp
from precision_attention_nvfp4_b200 import _lib

PTR = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from precision_attention_nvfp4_b200 import build
    build.build()
    return fp.library()


def accepted(lib, B, T, H, group, max_pages, page=128, d=128, start=False, num_pages=4):
    """Whether fpattn_cache_attention takes a call of these sizes (a workspace size of 0 is its refusal)."""
    hq = H * group
    q = _lib.Rows(PTR, 1 if start else B, B * T if start else T, hq, d, 0 if start else T * hq * d, hq * d, d)
    c = _lib.KvCache(PTR, PTR, PTR, num_pages, H, page, d)
    a = _lib.CacheQueries(q, PTR if start else None, B, T, PTR, max_pages, max_pages, PTR, 1, None, 0, 0, 0.0)
    need = lib.fpattn_cache_attention_workspace(ctypes.byref(c), ctypes.byref(a))
    st = lib.fpattn_cache_attention(ctypes.byref(c), ctypes.byref(a), PTR, None, None, 0, None)  # no workspace: no launch
    assert st == (_lib.ERR_INVALID_ARG if need else _lib.ERR_UNSUPPORTED)
    return need > 0


@pytest.mark.parametrize("start", [False, True])
def test_work_is_counted_in_the_tiles_that_run(lib, start):
    # 64 sequences, 8 KV heads, 1024 queries of group 4, a table of 2^20 tokens: 32 tiles of 128 rows a problem
    assert accepted(lib, 64, 1024, 8, 4, 1 << 13, start=start)
    # B * H * tiles of rows * (tiles of keys + 6) = 512 * 32 * 65536 = 2^30, and a tile of keys more
    assert accepted(lib, 64, 1024, 8, 4, 65530, start=start)
    assert not accepted(lib, 64, 1024, 8, 4, 65531, start=start)
    # one token: 16 rows a tile, a start of 8
    assert accepted(lib, 2048, 1, 8, 4, 65528, start=start)
    assert not accepted(lib, 2048, 1, 8, 4, 65529, start=start)
    # 32 and 33 rows a KV head: one tile each
    assert accepted(lib, 2048, 8, 8, 4, 65528, start=start)
    assert accepted(lib, 2048, 11, 8, 3, 65530, start=start)
    assert not accepted(lib, 2048, 11, 8, 3, 65531, start=start)


def test_other_limits(lib):
    assert accepted(lib, 1, 1, 1, 1, 1 << 23) and not accepted(lib, 1, 1, 1, 1, (1 << 23) + 1)      # 2^30 keys
    assert accepted(lib, 1, 1, 4096, 1, 4) and not accepted(lib, 1, 1, 4097, 1, 4)                  # KV heads
    assert accepted(lib, 1, 1, 2, 1, 4, num_pages=(1 << 30) - 1) and not accepted(lib, 1, 1, 2, 1, 4, num_pages=1 << 30)
    assert accepted(lib, 1 << 24, 1, 1, 1, 1) and not accepted(lib, (1 << 24) + 1, 1, 1, 1, 1)
    assert accepted(lib, 1, 1 << 20, 1, 1 << 8, 4) and not accepted(lib, 1, (1 << 20) + 1, 1, 1 << 8, 4)  # 2^28 rows
