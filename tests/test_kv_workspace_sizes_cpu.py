"""The workspace of attention over a cache: 0 for every size that the call refuses, and a sum that does not overflow
at the largest ones that it takes."""
import ctypes
import os

import pytest

import micro_scaled_fp4_amd as m

pytestmark = pytest.mark.skipif(not os.path.exists(m.LIB_PATH), reason="libfp4.so not built")


def size(T, B, q_heads, heads=2, dim=64, page=16, pages=4):
    held = m._KVCacheStruct(0, heads, dim, page, pages, 4096, 4096, 4096, 4096, 4096, 4096)
    return m.load_library().kv_cache_attention_workspace_bytes(ctypes.addressof(held), T, B, q_heads)


@pytest.mark.parametrize("T,q_heads", [(1 << 24, 128), (1 << 24, 1 << 16), (1 << 15, (1 << 15) + 2), (16400, 1 << 16)])
def test_more_query_rows_than_the_call_takes(T, q_heads):
    assert size(T, 1, q_heads) == 0


def test_caches_that_the_calls_refuse():
    assert size(4, 2, 4) > 0
    for bad in (dict(heads=0), dict(heads=2048, q_heads=2048), dict(dim=48), dict(dim=288), dict(page=24), dict(page=8), dict(page=1 << 17),
                dict(pages=-1), dict(pages=1 << 31), dict(T=0), dict(B=0), dict(T=(1 << 24) + 1), dict(B=(1 << 16) + 1), dict(q_heads=0),
                dict(q_heads=3)):
        assert size(**{**dict(T=4, B=2, q_heads=4), **bad}) == 0, bad


def test_largest_sizes():
    """At least the tiles' records (32 bytes each), and not past 2 GB beyond them."""
    for T, q_heads, heads in ((1 << 24, 64, 1), (1 << 24, 64, 64), (1 << 14, 1 << 16, 1), (1 << 14, 1 << 16, 1024), (1 << 24, 1, 1)):
        group = q_heads // heads
        least = 32 * (T * group // 128)
        got = size(T, 1 << 16, q_heads, heads, 256)
        assert least <= got <= 32 * (T * group // 16 + (1 << 17)) + (1 << 31), (T, q_heads, heads, got)
