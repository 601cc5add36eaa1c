"""Gathers and attention still queued on another stream, behind work that keeps
it busy, when the pool's own stream changes what they read; and attention to
the rows of a union list that a resolve has made."""
import pytest
import torch

from test_gpu_attend import LAYOUTS, Layout, compare
from test_gpu_fork import Env, dhs  # noqa: F401

pytestmark = pytest.mark.gpu
LAY = Layout(4, 24, 24)  # Env's rows of 24 elements


def busy(stream):
    """About 70 ms of work."""
    with torch.cuda.stream(stream):
        a = torch.randn(8192, 8192, device="cuda", dtype=torch.bfloat16)
        for _ in range(100):
            a = (a @ a).clamp(-1, 1)
    return a


class Reads:
    """A gather of k selected rows of request r, attention to them, and
    attention to its whole history: the same calls into fresh outputs."""

    def __init__(self, dhs, env, r):  # noqa: F811
        self.dhs, self.env, self.r = dhs, env, r
        self.sel = env.select(r)[0, :1]
        self.loc = torch.empty_like(self.sel)
        env.step += 1
        st, keep = dhs.make_step(env.step, [self.item(None)])
        assert env.pool.resolve(st) == 0
        self.q = torch.randn(1, LAY.heads, LAY.key, generator=env.g, device="cuda").bfloat16()

    def item(self, staging):
        it = self.dhs.dhs_item()
        it.req, it.queries, it.topk = self.r, 1, self.env.k
        it.sel_dev, it.loc_dev = self.sel.data_ptr(), self.loc.data_ptr()
        it.staging_dev = None if staging is None else staging.data_ptr()
        return it

    def enqueue(self, stream):
        """Through the calls for other streams, or (None) on the pool's own."""
        d, pool, k = self.dhs, self.env.pool, self.env.k
        staging = torch.zeros(k, self.env.E, dtype=torch.int16, device="cuda")
        out = torch.zeros(2, 1, LAY.heads, LAY.value, dtype=torch.bfloat16, device="cuda")
        items = [d.attend_item(queries=1, topk=k, q=self.q, loc=self.loc, out=out[0]),
                 d.attend_item(req=self.r, queries=1, q=self.q, out=out[1],
                               flags=d.DHS_ATTEND_HISTORY)]
        at, keep1 = d.make_attend(items, **LAY.args())
        work = torch.empty(max(256, pool.attend_bytes(at)), dtype=torch.uint8, device="cuda")
        at.work_dev, at.work_bytes = work.data_ptr(), work.numel()
        st, keep2 = d.make_step(self.env.step, [self.item(staging)])
        torch.cuda.synchronize()  # the buffers are ready on every stream
        block = None
        if stream is None:
            assert pool.gather(st) == 0 and pool.attend(at) == 0
        else:
            block = busy(stream)
            assert d.lib.dhs_gather_on(pool.h, d.ctypes.byref(st), stream.cuda_stream) == 0
            assert pool.attend_on(at, stream.cuda_stream) == 0
        return staging, out, (work, block)


def filled(env, r, n, resident):
    """Request r admitted with finite rows."""
    rows = torch.randn(1, env.max_rows, env.E, generator=env.g, device="cuda").bfloat16().view(torch.int16)
    mask = [1 if (i * 7) % 10 < 10 * resident else 0 for i in range(n // env.PR)]
    assert env.pool.admit_device(r, 0, rows.data_ptr(), env.host[r, 0].data_ptr(), n, mask)[0] == 0
    env.rows[r], env.len[r], env.n[r], env.window = rows, n, n, ()


@pytest.mark.parametrize("change", ["admit", "fork", "compact", "append", "reclaim"])
def test_reads_on_another_stream_come_first(dhs, change):  # noqa: F811
    n = 640
    env = Env(dhs, R=4, S=1, n=n, pages=130)
    for r in range(3):
        filled(env, r, n, 1.0)
    r = 2 if change == "compact" else 0
    reads = Reads(dhs, env, r)
    want = reads.enqueue(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = reads.enqueue(side)
    assert not side.query()  # still busy: what follows is queued behind it
    if change == "admit":
        assert env.pool.release(0) == 0
        filled(env, 3, n, 1.0)  # into the freed slots
        assert env.pool.flush() == 0
    elif change == "fork":
        assert env.pool.release(0) == 0
        assert env.pool.fork(1, 0, env.hosts(0))[0] == 0
    elif change == "compact":
        assert env.pool.release(0) == 0
        assert env.pool.compact(env.pool.used()) == (0, n // env.PR)
        env.pool.opt.view(-1, env.PR * env.E * 2)[env.pool.capacity():] = 0x5A  # lent out
    elif change == "append":
        for _ in range(3):
            env.append([0], env.T)  # the whole ring, three times
    else:
        assert env.pool.reclaim([0], n // env.PR)[0] == 0
        filled(env, 3, n, 1.0)
        assert env.pool.flush() == 0
    torch.cuda.synchronize()
    for a, b in zip(got[:2], want[:2]):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert env.pool.status() == (0, 0)


def test_refill_behind_attention_on_another_stream(dhs):  # noqa: F811
    """A refill that a later call flushes while the attention waits to run."""
    n = 640
    env = Env(dhs, R=2, S=1, n=n, pages=60)
    filled(env, 0, n, 0.3)
    filled(env, 1, n, 0.0)
    reads = Reads(dhs, env, 0)
    want = reads.enqueue(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = reads.enqueue(side)
    assert not side.query()
    assert env.pool.refill(100)[1] > 20
    st, keep = dhs.make_attend([], **LAY.args())
    assert env.pool.attend(st) == 0  # flushes
    after = reads.enqueue(None)
    torch.cuda.synchronize()
    for x in (got, after):
        for a, b in zip(x[:2], want[:2]):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("Q,k", [(1, 40), (4, 150), (8, 260)])
def test_union_list_of_a_resolve(dhs, Q, k):  # noqa: F811
    """Resolve a verify block into a union list, attend through its positions."""
    lay, n, T = LAYOUTS["latent"], 2000, 64
    g = torch.Generator("cuda").manual_seed(Q)
    pool = dhs.Pool(max_requests=1, sources=1, row_bytes=lay.elems * 2, page_rows=16, tail_rows=T,
                    hot_rows=2048, max_queries=8, max_topk=300, max_rows_per_request=n,
                    optional_pages=n // 16)
    rows = torch.randn(n, lay.elems, generator=g, device="cuda").bfloat16()
    host = torch.zeros(n, lay.elems, dtype=torch.bfloat16).pin_memory()
    mask = [i % 3 > 0 for i in range(n // 16)]
    assert pool.admit_device(0, 0, rows.data_ptr(), host.data_ptr(), n, mask)[0] == 0
    for step in (1, 2):  # the second one finds its rows in the hot cache
        shared = torch.randperm(n, generator=g, device="cuda")[:k]
        sel = shared.repeat(Q, 1)  # three quarters in common, each in its own order
        for i in range(Q):
            sel[i, k - k // 4:] = torch.randint(0, n, (k // 4,), generator=g, device="cuda")
            sel[i] = sel[i][torch.randperm(k, generator=g, device="cuda")]
        sel = sel.int().contiguous()
        loc, index = torch.empty_like(sel), torch.empty_like(sel)
        it = dhs.dhs_item()
        it.queries, it.topk, it.flags = Q, k, dhs.DHS_ITEM_UNION
        it.sel_dev, it.loc_dev, it.index_dev = sel.data_ptr(), loc.data_ptr(), index.data_ptr()
        st, keep = dhs.make_step(step, [it])
        assert pool.resolve(st) == 0
        q = torch.randn(Q, lay.heads, lay.key, generator=g, device="cuda").bfloat16()
        out = torch.empty(Q, lay.heads, lay.value, dtype=q.dtype, device="cuda")
        lse = torch.empty(Q, lay.heads, device="cuda")
        at, keep2 = dhs.make_attend([dhs.attend_item(queries=Q, topk=k, q=q, loc=loc, index=index,
                                                     out=out, lse=lse)], **lay.args())
        work = torch.empty(max(256, pool.attend_bytes(at)), dtype=torch.uint8, device="cuda")
        at.work_dev, at.work_bytes = work.data_ptr(), work.numel()
        assert pool.attend(at) == 0 and pool.status() == (0, 0)
        compare(lay, q, rows[sel.long()], torch.ones(Q, k, dtype=torch.bool, device="cuda"), out, lse)
    pool.close()
