"""Forks whose parent has fewer sources than the child's slot held before: the
slot's old pages are gone for every reader of the pool's maps."""
import pytest
import torch

from test_gpu_attend import Layout, compare, run
from test_gpu_fork import Env, dhs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("parent_src", [0, 1])
@pytest.mark.parametrize("fused", [False, True])
def test_source_that_the_parent_lacks(dhs, parent_src, fused):  # noqa: F811
    n, other = 320, 1 - parent_src
    env = Env(dhs, R=3, S=2, n=n, pages=60)
    rows = torch.randn(3, n, env.E, generator=env.g, device="cuda").bfloat16()  # parent, old, new

    def admit(r, s, x, resident):
        rc, _ = env.pool.admit_device(r, s, x.data_ptr(), env.host[r, s].data_ptr(), n,
                                      [resident] * (n // env.PR))
        assert rc == 0

    admit(0, parent_src, rows[0], 1)
    for s in range(2):
        admit(1, s, rows[1], 1)
    assert env.pool.flush() == 0 and env.pool.release(1) == 0
    assert env.pool.fork(0, 1, env.hosts(1))[0] == 0
    admit(1, other, rows[2], 0)  # no resident page
    want = {parent_src: rows[0], other: rows[2]}
    # resolve and gather
    sel = torch.randint(0, n, (2, 1, env.k), generator=env.g, device="cuda").int()
    loc, stg = torch.empty_like(sel), torch.empty(2, 1, env.k, env.E, dtype=rows.dtype, device="cuda")
    items = []
    for s in range(2):
        it = dhs.dhs_item()
        it.req, it.src, it.queries, it.topk = 1, s, 1, env.k
        it.sel_dev, it.loc_dev, it.staging_dev = sel[s].data_ptr(), loc[s].data_ptr(), stg[s].data_ptr()
        items.append(it)
    st, keep = dhs.make_step(1, items)
    if fused:
        assert env.pool.resolve_gather(st) == 0
    else:
        assert env.pool.resolve(st) == 0 and env.pool.gather(st) == 0
    assert env.pool.status() == (0, 0)
    for s in range(2):
        assert torch.equal(stg[s, 0], want[s][sel[s, 0].long()])
    # history attention
    lay = Layout(4, env.E, env.E)
    q = torch.randn(2, 1, 4, env.E, generator=env.g, device="cuda").bfloat16()
    out, lse = torch.empty_like(q), torch.empty(2, 1, 4, device="cuda")
    run(dhs, env.pool, lay, [dhs.attend_item(req=1, src=s, queries=1, q=q[s], out=out[s], lse=lse[s],
                                             flags=dhs.DHS_ATTEND_HISTORY) for s in range(2)])
    torch.cuda.synchronize()
    for s in range(2):
        compare(lay, q[s], want[s][None], torch.ones(1, n, dtype=torch.bool, device="cuda"),
                out[s], lse[s])
