"""Arenas that a caller hands to a pool: memory of another device is refused
before any kernel can be given its address."""
import pytest


@pytest.mark.parametrize("count", [1, 2, 3])
def test_arena_of_another_device(count):
    torch = pytest.importorskip("torch")
    from hierarchical_sparse_kv_dhs_gb300.build import build
    build()
    from hierarchical_sparse_kv_dhs_gb300 import dhs
    size = dict(max_requests=1, sources=1, row_bytes=16, page_rows=16, tail_rows=4, hot_rows=4,
                max_queries=1, max_topk=1, max_rows_per_request=64, optional_pages=4)
    arenas = [torch.empty(4096, dtype=torch.uint8) for _ in range(count)]
    with pytest.raises(ValueError, match="cuda:0"):
        dhs.Pool(device="cuda:0", stream=object(), arenas=arenas, **size)
