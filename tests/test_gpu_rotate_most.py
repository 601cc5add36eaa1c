"""A rotation of as many tokens as its step can name."""
import pytest
import torch

from test_gpu_packed_rows import dhs, frequencies, pool_of, turned  # noqa: F401

pytestmark = pytest.mark.gpu


def test_rotate_as_many_tokens_as_there_can_be(dhs):  # noqa: F811
    """2^31 - 1 tokens (69 GB of results), one head that all of them share on the way in."""
    n = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB of device memory")
    x = torch.randn(1, 1, 16, device="cuda").half()
    at = torch.arange(n, dtype=torch.int32, device="cuda")
    out = torch.empty(n, 1, 16, dtype=torch.float16, device="cuda")
    for i in range(0, n, 1 << 24):  # the ends of what a chunk of blocks writes
        out[i:i + 2] = 7
    out[-2:] = 7
    table = torch.from_numpy(dhs.rope_table(16)).cuda()
    pool = pool_of(dhs)
    assert pool.rotate(dhs.make_rotate(x.expand(n, 1, 16), at, table, out=out)) == 0
    torch.cuda.synchronize()
    some = torch.cat([torch.arange(0, n, 999983, device="cuda"), torch.arange(n - 600, n, device="cuda")] +
                     [torch.arange(i, i + 2, device="cuda") for i in range(0, n, 1 << 24)])
    want, m = turned(x.expand(len(some), 1, 16), some, frequencies(16), "half")
    # far positions: the bound of the test of far positions
    assert bool(((out[some].double() - want).abs() <= 2.0 ** -18 * m + 1.01 * 2.0 ** -11 * want.abs() + 2.0 ** -25).all())
    del out, at
    torch.cuda.empty_cache()
