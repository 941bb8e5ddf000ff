"""GPU: out_dtype beside an out of another type is refused by the cache calls, not ignored."""
import pytest
import torch

import micro_scaled_fp4_amd as fp4
from gpu_util import DEV, announce
from test_gpu_kv_cache import i32

pytestmark = pytest.mark.gpu


def test_out_dtype_and_out():
    announce("kv cache out_dtype beside out")
    T, H, D = 5, 2, 64
    cache = fp4.KVCache.empty(fp4.FP4_MXFP4, 1, H, 16, D, device=DEV)
    x = torch.randn(T, H, D, device=DEV)
    where = i32([0, T]), i32([T]), i32([[0]])
    fp4.kv_cache_write(cache, x, x, *where)
    other = {torch.float32: torch.bfloat16, torch.bfloat16: torch.float32}
    for dtype in other:
        k, v, y = (torch.full((T, H, D), 9.0, dtype=dtype, device=DEV) for _ in range(3))
        with pytest.raises(TypeError):
            fp4.kv_cache_read(cache, *where, T, out_dtype=other[dtype], out=(k, v))
        with pytest.raises(TypeError):
            fp4.kv_cache_attention(cache, x, *where, out_dtype=other[dtype], out=y)
        assert all((t == 9.0).all() for t in (k, v, y))
        for kind in (None, dtype):              # out's own type, named or not
            got = fp4.kv_cache_read(cache, *where, T, out_dtype=kind, out=(k, v))
            assert got[0] is k and got[1] is v
            assert fp4.kv_cache_attention(cache, x, *where, out_dtype=kind, out=y) is y
        want = fp4.kv_cache_read(cache, *where, T, out_dtype=dtype)
        assert isinstance(want, tuple) and torch.equal(k, want[0]) and torch.equal(v, want[1])
        assert torch.equal(y, fp4.kv_cache_attention(cache, x, *where, out_dtype=dtype))
    assert fp4.kv_cache_read(cache, *where, T)[0].dtype == torch.bfloat16
    assert fp4.kv_cache_attention(cache, x, *where).dtype == torch.float32
