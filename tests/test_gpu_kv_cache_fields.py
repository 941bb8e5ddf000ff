"""GPU: a cache's tensors are changed in place, and the calls see it."""
import pytest
import torch

import micro_scaled_fp4_amd as fp4
from gpu_util import DEV, announce
from test_gpu_kv_cache import i32

pytestmark = pytest.mark.gpu


def test_an_amax_changed_in_place():
    announce("kv cache amax changed in place")
    T, H, D = 20, 2, 64
    x = torch.randn(T, H, D, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    where = i32([0, T]), i32([T]), i32([[1, 0]])
    cache, other = (fp4.KVCache.empty(fp4.FP4_NVFP4, 2, H, 16, D, a, 2.0, device=DEV) for a in (3.0, 7.0))
    held = cache.k_amax
    with pytest.raises(AttributeError):
        cache.k_amax = torch.full((1,), 7.0, device=DEV)
    assert cache.k_amax is held
    cache.k_amax.fill_(7.0)
    for c in (cache, other):
        fp4.kv_cache_write(c, x, x, *where)
    for a, b in zip(fp4.kv_cache_read(cache, *where, T), fp4.kv_cache_read(other, *where, T)):
        assert torch.equal(a, b)
    assert torch.equal(fp4.kv_cache_attention(cache, x, *where), fp4.kv_cache_attention(other, x, *where))
