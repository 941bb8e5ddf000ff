"""A KVCache's fields cannot be replaced: the library reads the addresses that it was made with."""
import copy
import ctypes
import os

import pytest

import micro_scaled_fp4_amd as m


def made():
    """A cache as its constructor leaves it, without a device."""
    c = object.__new__(m.KVCache)
    for name in m.KVCache.__slots__:
        if name not in ("_struct", "_address"):
            setattr(c, name, name)
    c._struct = m._KVCacheStruct(0, 2, 64, 16, 4, 4096, 4096, 4096, 4096, 4096, 4096)
    c._address = ctypes.addressof(c._struct)
    return c


@pytest.mark.skipif(not os.path.exists(m.LIB_PATH), reason="libfp4.so not built")
@pytest.mark.parametrize("name", m.KVCache.__slots__)
def test_fields_are_not_replaced(name):
    c = made()
    before = getattr(c, name)
    with pytest.raises(AttributeError):
        setattr(c, name, 0)
    with pytest.raises(AttributeError):
        delattr(c, name)
    assert getattr(c, name) is before


@pytest.mark.skipif(not os.path.exists(m.LIB_PATH), reason="libfp4.so not built")
def test_copies_and_subclasses():
    c = made()
    other = copy.copy(c)
    assert all(getattr(other, name) is getattr(c, name) for name in m.KVCache.__slots__)
    with pytest.raises(AttributeError):
        other.k_codes = 0

    class Named(m.KVCache):
        pass

    n = Named.__new__(Named)
    for name in m.KVCache.__slots__:
        setattr(n, name, getattr(c, name))
    n.layer = 3
    n.layer = 4
    del n.layer
    with pytest.raises(AttributeError):
        n.v_codes = 0
