"""The attention, fork and compaction entry points without a GPU: null pools
and steps are refused before any device work."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def dhs():
    from hierarchical_sparse_kv_dhs_gb300.build import build
    build()
    from hierarchical_sparse_kv_dhs_gb300 import dhs as mod
    return mod


def test_null_arguments(dhs):
    E = dhs.DHS_EINVAL
    n64, size = ctypes.c_int64(0), ctypes.c_size_t(0)
    st, keep = dhs.make_attend([], heads=1, key_elems=8, value_elems=8, scale=1.0)
    assert dhs.lib.dhs_attend(None, ctypes.byref(st)) == E
    assert dhs.lib.dhs_attend(None, None) == E
    assert dhs.lib.dhs_attend_on(None, ctypes.byref(st), 1) == E
    assert dhs.lib.dhs_attend_bytes(None, ctypes.byref(st), ctypes.byref(size)) == E
    assert dhs.lib.dhs_attend_bytes(None, ctypes.byref(st), None) == E
    assert dhs.lib.dhs_fork(None, 0, 1, None, None, ctypes.byref(n64)) == E
    assert dhs.lib.dhs_compact(None, 0, ctypes.byref(n64)) == E
    assert dhs.lib.dhs_pool_capacity(None) == -1


def test_descriptors_match_the_header(dhs):
    """The ctypes structures have the C ones' sizes (LP64: no hidden padding)."""
    assert ctypes.sizeof(dhs.dhs_attend_item) == 6 * 4 + 6 * 8
    assert ctypes.sizeof(dhs.dhs_attend_step) == 12 * 4 + 4 * 8 + 3 * 8


def test_pool_refuses_short_arenas(dhs):
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        dhs.Pool(max_requests=1, sources=1, row_bytes=16, page_rows=16, tail_rows=4, hot_rows=4,
                 max_queries=1, max_topk=1, max_rows_per_request=64, optional_pages=4,
                 device="cuda:0", stream=object(), arenas=(torch.empty(8, dtype=torch.uint8),))
