"""The binding declares the argument types of every function in the header.  An
undeclared one takes a pool's handle as a C int, which cuts off the upper half
of the address and crashes wherever the heap lies above 2 GiB."""
import ctypes

import pytest

from test_abi import declared_functions, dhs  # noqa: F401


@pytest.mark.parametrize("name", declared_functions())
def test_argument_types_are_declared(dhs, name):  # noqa: F811
    f = getattr(dhs.lib, name)
    assert f.argtypes is not None and len(f.argtypes) > 0
    if name in ("dhs_pool_bytes", "dhs_strerror"):
        return
    if name == "dhs_pool_create":
        assert f.argtypes[1] is ctypes.POINTER(ctypes.c_void_p)
    else:
        assert f.argtypes[0] is ctypes.c_void_p  # the pool
