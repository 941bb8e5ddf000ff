"""Host-side checks of the cache calls (no GPU needed): bad arguments come back as their status before
anything reaches a device, and the binding refuses wrong types, shapes and host tensors."""
import ctypes
import os

import pytest
import torch

import micro_scaled_fp4_amd as m

pytestmark = pytest.mark.skipif(not os.path.exists(m.LIB_PATH), reason="libfp4.so not built")

OK, NULL, SHAPE, DTYPE, ALIGN, ARCH, WORKSPACE, HIP, ALIAS = range(9)
P, Q, R = (ctypes.c_void_p(a) for a in (4096, 8192, 12288))     # never dereferenced
ODD = ctypes.c_void_p(4097)


def cache(fmt=0, heads=2, dim=64, page=16, pages=4, k=4096, ks=4096, v=4096, vs=4096, ka=4096, va=4096):
    if fmt == 1 and ka == 4096 and va == 4096:
        ka = va = None
    return m._KVCacheStruct(fmt, heads, dim, page, pages, k, ks, v, vs, ka, va)


def write(c, k=P, ks=128, v=P, vs=128, t=1, T=4, B=2, off=P, ln=P, pg=P, wide=3):
    return m.load_library().kv_cache_write(c and ctypes.addressof(c), k, ks, v, vs, t, T, B, off, ln, pg, wide, None)


def read(c, T=4, B=2, off=P, st=None, ln=P, pg=P, wide=3, k=P, v=Q, t=1):
    return m.load_library().kv_cache_read(c and ctypes.addressof(c), T, B, off, st, ln, pg, wide, k, v, t, None)


def attend(c, q=P, qs=256, qt=1, T=4, heads=4, B=2, off=P, ln=P, pg=P, wide=3, scale=1.0, causal=1, window=0, out=Q, ot=1, lse=None,
           ws=P, n=1 << 40):
    return m.load_library().kv_cache_attention(c and ctypes.addressof(c), q, qs, qt, T, heads, B, off, ln, pg, wide, scale, causal,
                                               window, out, ot, lse, ws, n, None)


@pytest.mark.parametrize("call", [write, read, attend])
def test_shared_argument_errors(call):
    assert call(None) == NULL
    assert call(cache(fmt=2)) == DTYPE and call(cache(fmt=-1)) == DTYPE
    assert call(cache(heads=0)) == SHAPE and call(cache(heads=1025)) == SHAPE
    for dim in (0, 16, 48, 288, -32):
        assert call(cache(dim=dim)) == SHAPE
    for page in (0, 8, 24, 48, 1 << 17, -16):
        assert call(cache(page=page)) == SHAPE
    assert call(cache(pages=-1)) == SHAPE and call(cache(pages=1 << 31)) == SHAPE
    assert call(cache(), T=-1) == SHAPE and call(cache(), T=(1 << 24) + 1) == SHAPE
    assert call(cache(), B=-1) == SHAPE and call(cache(), B=(1 << 16) + 1) == SHAPE
    assert call(cache(), wide=-1) == SHAPE and call(cache(), wide=(1 << 26) + 1) == SHAPE
    assert call(cache(fmt=1, ka=4096, va=None)) == DTYPE
    assert call(cache(ka=None)) == NULL and call(cache(va=None)) == NULL
    assert call(cache(), off=None) == NULL and call(cache(), ln=None) == NULL and call(cache(), pg=None) == NULL
    for name in ("k", "ks", "v", "vs"):
        assert call(cache(**{name: None})) == NULL
        assert call(cache(**{name: 4104})) == ALIGN
    assert call(cache(ka=4098)) == ALIGN and call(cache(va=4098)) == ALIGN
    assert call(cache(), off=ODD) == ALIGN and call(cache(), ln=ODD) == ALIGN and call(cache(), pg=ODD) == ALIGN
    assert call(cache(), T=0) == OK and call(cache(), B=0) == OK
    assert call(cache(fmt=1), T=0, off=None, ln=None, pg=None) == OK


def test_write_argument_errors():
    assert write(cache(), t=2) == DTYPE
    assert write(cache(), ks=-1) == SHAPE and write(cache(), vs=-1) == SHAPE and write(cache(), ks=1 << 40) == SHAPE
    assert write(cache(), k=None) == NULL and write(cache(), v=None) == NULL
    assert write(cache(), k=ODD) == ALIGN and write(cache(), v=ctypes.c_void_p(4098), t=0) == ALIGN


def test_read_argument_errors():
    assert read(cache(), t=2) == DTYPE
    assert read(cache(), k=None) == NULL and read(cache(), v=None) == NULL
    assert read(cache(), k=ODD) == ALIGN and read(cache(), st=ODD) == ALIGN
    assert read(cache(), v=P) == ALIAS


def test_attention_argument_errors():
    assert attend(cache(), qt=2) == DTYPE and attend(cache(), ot=2) == DTYPE
    assert attend(cache(), heads=0) == SHAPE and attend(cache(), heads=3) == SHAPE and attend(cache(), heads=(1 << 16) + 2) == SHAPE
    assert attend(cache(), T=1 << 24, heads=128) == SHAPE
    assert attend(cache(), qs=-1) == SHAPE and attend(cache(), window=-1) == SHAPE
    assert attend(cache(), window=5, causal=0) == SHAPE
    for scale in (float("inf"), float("nan"), -float("inf")):
        assert attend(cache(), scale=scale) == SHAPE
    assert attend(cache(), q=None) == NULL and attend(cache(), out=None) == NULL
    held = cache()
    need = m.load_library().kv_cache_attention_workspace_bytes(ctypes.addressof(held), 4, 2, 4)
    assert need > 0
    assert attend(cache(), ws=None) == WORKSPACE and attend(cache(), n=need - 1) == WORKSPACE
    assert attend(cache(), q=ODD) == ALIGN and attend(cache(), out=ODD) == ALIGN and attend(cache(), ws=ctypes.c_void_p(4100)) == ALIGN
    assert attend(cache(), lse=ODD) == ALIGN
    assert attend(cache(), out=P) == ALIAS and attend(cache(), lse=Q) == ALIAS


def test_workspace_of_bad_sizes_is_zero():
    f = m.load_library().kv_cache_attention_workspace_bytes
    held = cache()
    c = ctypes.addressof(held)
    assert f(None, 4, 2, 4) == 0 and f(c, 0, 2, 4) == 0 and f(c, 4, 0, 4) == 0 and f(c, 4, 2, 3) == 0 and f(c, 4, 2, 0) == 0


def test_binding_refuses_host_tensors():
    z = torch.zeros(2, 2, 16, 32, dtype=torch.uint8)
    s = torch.zeros(2, 2, 16, 4, dtype=torch.uint8)
    with pytest.raises(ValueError):
        m.KVCache(m.FP4_NVFP4, z, s, z, s, 1.0, 1.0)
    with pytest.raises(ValueError):
        m.KVCache(7, z, s, z, s)
    with pytest.raises(ValueError):
        m.KVCache(m.FP4_MXFP4, z[0], s, z, s)


def test_binding_checks_before_the_library():
    """Shapes and types of the sequences' tensors and of rows (host tensors standing in: the first check that
    looks at the device comes after them)."""
    class Stub:
        device, num_heads, head_dim = torch.device("cpu"), 2, 64

    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    assert m._sequences(Stub, i(4), i(3), i(3, 5))[0::4] == (3, 5)
    for bad in ((i(3), i(3), i(3, 5)), (i(4), i(3), i(2, 5)), (i(4), i(3), i(15)), (i(4), i(3, 1), i(3, 5)), (i(4, 1), i(3), i(3, 5))):
        with pytest.raises(ValueError):
            m._sequences(Stub, *bad)
    for bad in ((i(4).long(), i(3), i(3, 5)), (i(4), i(3).float(), i(3, 5)), (i(4), i(3), i(3, 5).to(torch.int16))):
        with pytest.raises(TypeError):
            m._sequences(Stub, *bad)
    rows = torch.zeros(5, 9, 64)
    t, stride = m._head_rows(rows[:, 2:4], 2, 64, Stub.device, "k")
    assert t.data_ptr() == rows[:, 2:4].data_ptr() and stride == 9 * 64
    t, stride = m._head_rows(torch.zeros(2, 5, 64).transpose(0, 1), 2, 64, Stub.device, "k")
    assert t.is_contiguous() and stride == 128
    t, stride = m._head_rows(torch.zeros(1, 2, 64).expand(5, 2, 64), 2, 64, Stub.device, "k")
    assert stride == 0
    for bad in (torch.zeros(5, 128), torch.zeros(5, 3, 64), torch.zeros(5, 2, 32)):
        with pytest.raises(ValueError):
            m._head_rows(bad, 2, 64, Stub.device, "k")
