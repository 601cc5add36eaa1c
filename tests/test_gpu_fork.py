"""dhs_fork and dhs_compact: copies are bit-exact, so every comparison here is
for equality.  A fork must behave as its parent from then on: the same steps
give the same counters, tiers, staged bytes, tags and stamps."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dhs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from hierarchical_sparse_kv_dhs_gb300.build import build
    build()
    from hierarchical_sparse_kv_dhs_gb300 import dhs as mod
    return mod


class Env:
    """A pool whose rows are known: rows[r][s] holds request r's rows."""

    def __init__(self, dhs, R=3, S=2, n=1000, PR=16, T=24, B=120, E=24, pages=400, k=40, seed=0,
                 reserve=0, max_rows=None):
        self.dhs, self.S, self.PR, self.T, self.B, self.E, self.k = dhs, S, PR, T, B, E, k
        self.g = torch.Generator("cuda").manual_seed(seed)
        self.max_rows = max_rows or n + 400
        self.pool = dhs.Pool(max_requests=R, sources=S, row_bytes=E * 2, page_rows=PR, tail_rows=T,
                             hot_rows=B, max_queries=2, max_topk=k, max_rows_per_request=self.max_rows,
                             optional_pages=pages, admission_reserve_pages=reserve)
        self.host = torch.zeros(R, S, self.max_rows, E, dtype=torch.int16).pin_memory()
        self.rows, self.len, self.n, self.step = {}, {}, {}, 0

    def admit(self, r, n, resident=0.5, window=()):
        rows = torch.randint(-30000, 30000, (self.S, self.max_rows, self.E), generator=self.g,
                             device="cuda").to(torch.int16)
        for s in range(self.S):
            if s in window:
                m = min(n, self.T)
                rc = self.pool.admit_window(r, s, rows[s, n - m:].data_ptr(), n)
            else:
                mask = torch.rand(n // self.PR, generator=self.g, device="cuda") < resident
                rc, deficit = self.pool.admit_device(r, s, rows[s].data_ptr(),
                                                     self.host[r, s].data_ptr(), n, mask.cpu().numpy())
            assert rc == 0, (rc, s)
        self.rows[r], self.len[r], self.n[r] = rows, n, n
        self.window = window

    def hosts(self, r):
        return [self.host[r, s].data_ptr() for s in range(self.S)]

    def fork(self, r, child, masks=None, expect=0):
        rc, deficit = self.pool.fork(r, child, self.hosts(child), masks)
        assert rc == expect, rc
        if rc == 0:
            self.rows[child] = self.rows[r].clone()
            self.len[child], self.n[child] = self.len[r], self.n[r]
        return deficit

    def append(self, rs, count):
        items = []
        for r in rs:
            for s in range(self.S):
                a = self.dhs.dhs_append_item()
                a.req, a.src, a.count = r, s, count
                a.rows_dev = self.rows[r][s, self.len[r]].data_ptr()
                items.append(a)
            self.len[r] += count
        assert self.pool.append(items) == 0

    def select(self, r):
        """Random rows [S][2][k] of the request (a window source: of its window)."""
        out = torch.empty(self.S, 2, self.k, dtype=torch.int32, device="cuda")
        for s in range(self.S):
            lo = max(0, self.len[r] - self.T) if s in self.window else 0
            out[s] = torch.randint(lo, self.len[r], (2, self.k), generator=self.g, device="cuda")
        return out

    def decode(self, sels):
        """One step: {request: selection}; returns {request: (loc, counters, staging)}."""
        self.step += 1
        items, out = [], {}
        for r, sel in sels.items():
            loc = torch.empty(self.S, 2, self.k, dtype=torch.int32, device="cuda")
            cnt = torch.empty(self.S, 8, dtype=torch.int32, device="cuda")
            stg = torch.empty(self.S, 2, self.k, self.E, dtype=torch.int16, device="cuda")
            for s in range(self.S):
                it = self.dhs.dhs_item()
                it.req, it.src, it.queries, it.topk = r, s, 2, self.k
                it.sel_dev, it.loc_dev = sel[s].data_ptr(), loc[s].data_ptr()
                it.counters_dev, it.staging_dev = cnt[s].data_ptr(), stg[s].data_ptr()
                items.append(it)
            out[r] = (loc, cnt, stg)
        st, keep = self.dhs.make_step(self.step, items)
        assert self.pool.resolve_gather(st) == 0
        assert self.pool.status() == (0, 0)
        for r, sel in sels.items():
            want = torch.stack([self.rows[r][s][sel[s].long()] for s in range(self.S)])
            assert torch.equal(out[r][2], want), f"request {r}: staged rows"
        return out

    def state(self, r, s):
        return self.pool.read_state(r, s)

    def same_state(self, a, b, pages=True):
        for s in range(self.S):
            x, y = self.state(a, s), self.state(b, s)
            assert np.array_equal(x[0], y[0]) and np.array_equal(x[1], y[1])
            if pages:
                assert np.array_equal(x[2] >= 0, y[2] >= 0)
            assert np.array_equal(x[3][:3], y[3][:3])

    def same_step(self, a, b):
        sel = self.select(a)
        out = self.decode({a: sel, b: sel})
        for x, y in zip(out[a][1:], out[b][1:]):
            assert torch.equal(x, y)
        la, lb = out[a][0], out[b][0]
        assert torch.equal(la.long() >> 30 & 3, lb.long() >> 30 & 3)


@pytest.mark.parametrize("n,appended", [(1000, 0), (1000, 70), (15, 3), (16, 0), (5, 0), (0, 30), (160, 25)])
def test_fork_continues_as_its_parent(dhs, n, appended):
    env = Env(dhs, n=n)
    env.admit(0, n)
    for _ in range(appended):
        env.append([0], 1)
        env.decode({0: env.select(0)})
    if env.len[0]:
        env.decode({0: env.select(0)})
    env.fork(0, 2)
    env.same_state(0, 2)
    for i in range(6):
        env.append([0, 2], 3)  # the same rows on both sides
        env.same_step(0, 2)
        env.same_state(0, 2)
    # from here on they differ
    env.rows[2][:, env.len[2]:] += 1
    env.append([0, 2], 20)
    env.append([0, 2], 20)
    for i in range(4):
        env.decode({0: env.select(0), 2: env.select(2)})


def test_fork_of_a_fork_and_after_the_parent_is_gone(dhs):
    env = Env(dhs, n=500)
    env.admit(0, 500)
    env.append([0], 20)
    env.decode({0: env.select(0)})
    env.fork(0, 1)
    assert env.pool.release(0) == 0
    env.append([1], 24)
    env.decode({1: env.select(1)})
    env.fork(1, 0)
    assert env.pool.release(1) == 0
    # the freed pages are overwritten by another request
    env.admit(1, 480, resident=2.0)
    for _ in range(3):
        env.append([0], 10)
        env.decode({0: env.select(0), 1: env.select(1)})


def test_fork_with_masks_and_backup(dhs):
    """The child keeps fewer, other or more pages; its deferred backups are
    complete before its pages are taken."""
    env = Env(dhs, n=800)
    env.admit(0, 800, resident=0.5)
    P = 800 // env.PR
    r = np.random.default_rng(0)
    for masks in ([np.zeros(P), None], [np.ones(P), np.zeros(P)],
                  [r.integers(0, 2, P), r.integers(0, 2, P)]):
        pending = env.pool.pending_backup()
        env.fork(0, 1, masks)
        for s in range(2):
            have = env.state(1, s)[2][:P] >= 0
            want = env.state(0, s)[2][:P] >= 0 if masks[s] is None else masks[s] != 0
            assert np.array_equal(have, want)
        kept = int(sum((env.state(1, s)[2] >= 0).sum() for s in range(2)))
        assert env.pool.pending_backup() == pending + kept
        env.decode({1: env.select(1)})
        rc, freed = env.pool.reclaim([1], kept)
        assert rc == 0 and freed == kept and env.pool.pending_backup() == pending
        env.decode({1: env.select(1)})
        torch.cuda.synchronize()
        assert torch.equal(env.host[1, :, :800], env.rows[1][:, :800].cpu())
        assert env.pool.refill(1000)[0] == 0
        env.decode({1: env.select(1)})
        assert env.pool.release(1) == 0


def test_fork_of_pages_not_copied_yet(dhs):
    """Pages admitted from the host are still pending when the fork is made."""
    env = Env(dhs, n=400)
    rows = torch.randint(-30000, 30000, (2, env.max_rows, env.E), generator=env.g, device="cuda").to(torch.int16)
    env.host[0, :, :400] = rows[:, :400].cpu()
    for s in range(2):
        assert env.pool.admit(0, s, env.host[0, s].data_ptr(), 400)[0] == 0
    env.rows[0], env.len[0], env.n[0], env.window = rows, 400, 400, ()
    env.fork(0, 1)
    env.same_step(0, 1)


def test_fork_window_sources(dhs):
    for n in (0, 10, 24, 200):
        env = Env(dhs, S=2, n=200)
        env.admit(0, n, window=(1,))
        env.append([0], 5)
        env.fork(0, 1)
        for _ in range(3):
            env.append([0, 1], 7)
            env.same_step(0, 1)


def test_fork_many_sources(dhs):
    """More sources than one launch's table."""
    env = Env(dhs, R=2, S=260, n=40, T=4, B=8, E=8, pages=2 * 260 * 2, k=4)
    env.admit(0, 40, resident=2.0)
    env.decode({0: env.select(0)})
    env.fork(0, 1)
    env.same_state(0, 1)
    env.same_step(0, 1)


def test_fork_while_other_streams_read(dhs):
    """A gather on another stream and a prefetch are ordered before the fork."""
    env = Env(dhs, n=600)
    env.admit(0, 600)
    side = torch.cuda.Stream()
    sel = env.select(0)
    loc = torch.empty(2, 2, env.k, dtype=torch.int32, device="cuda")
    items = []
    for s in range(2):
        it = dhs.dhs_item()
        it.src, it.queries, it.topk = s, 2, env.k
        it.sel_dev, it.loc_dev = sel[s].data_ptr(), loc[s].data_ptr()
        items.append(it)
    env.step += 1
    st, keep = dhs.make_step(env.step, items)
    assert dhs.lib.dhs_prefetch(env.pool.h, dhs.ctypes.byref(st), side.cuda_stream) == 0
    env.fork(0, 1)
    env.same_state(0, 1)
    env.same_step(0, 1)


def test_fork_refusals(dhs):
    env = Env(dhs, n=320, pages=60, reserve=4)
    E, hosts = dhs.DHS_EINVAL, env.hosts(1)
    assert env.pool.fork(0, 1, hosts)[0] == dhs.DHS_ESTATE  # nothing there
    env.admit(0, 320, resident=2.0)  # 40 pages
    used = env.pool.used()

    def untouched():
        assert env.pool.used() == used and env.state(1, 0)[3][2] == 0 and env.state(1, 1)[3][2] == 0

    for a, b in ((0, 0), (-1, 1), (0, 3), (3, 1), (0, -1)):
        assert env.pool.fork(a, b, hosts)[0] == E
    assert env.pool.fork(0, 1, [hosts[0], 0])[0] == E
    assert env.pool.fork(0, 1, [hosts[0], hosts[1] + 8])[0] == E
    assert env.pool.fork(0, 1, env.hosts(0))[0] == E  # the parent's own rows
    plain = np.zeros(env.max_rows * env.E * 2 + 16, np.uint8)
    at = plain.ctypes.data + (-plain.ctypes.data) % 16
    # pageable memory: refused where the GPU cannot reach it
    assert env.pool.fork(0, 1, [hosts[0], at])[0] in (E, dhs.DHS_EWOULDWAIT)
    untouched()
    rc, deficit = env.pool.fork(0, 1, hosts)
    assert rc == dhs.DHS_EWOULDWAIT and deficit == 40 + 40 - 56
    untouched()
    half = [np.ones(20), np.zeros(20)]
    half[0][16:] = 0
    assert env.fork(0, 1, half) == 0
    assert env.pool.fork(0, 1, hosts)[0] == dhs.DHS_ESTATE
    assert env.pool.fork(2, 1, hosts)[0] == dhs.DHS_ESTATE
    env.decode({0: env.select(0), 1: env.select(1)})


# --------------------------------------------------------------- compaction

@pytest.mark.parametrize("seed", range(4))
def test_compact_keeps_every_page(dhs, seed):
    """Random admissions, releases and forks; after each compaction the pages
    lie in the lowest slots, every row reads as before, and memory past the
    capacity is the caller's."""
    env = Env(dhs, R=6, n=700, pages=300, seed=seed)
    r = np.random.default_rng(seed)
    live = set()
    for turn in range(14):
        free = [x for x in range(6) if x not in live]
        if free and (len(live) < 2 or r.random() < 0.6):
            x = int(r.choice(free))
            if live and r.random() < 0.4:
                p = int(r.choice(sorted(live)))
                if env.pool.fork(p, x, env.hosts(x))[0]:
                    continue
                env.rows[x], env.len[x], env.n[x] = env.rows[p].clone(), env.len[p], env.n[p]
            else:
                env.admit(x, int(r.integers(0, 300)), resident=0.6)
            live.add(x)
        elif live:
            x = int(r.choice(sorted(live)))
            assert env.pool.release(x) == 0
            live.discard(x)
        used = env.pool.used()
        cap = int(r.integers(used, 301))
        before = {(x, s): env.state(x, s)[2] for x in live for s in range(2)}
        rc, moved = env.pool.compact(cap)
        assert rc == 0 and env.pool.capacity() == cap and env.pool.used() == used
        slots, low, went = [], [], 0
        for key, old in before.items():
            new = env.state(*key)[2]
            assert np.array_equal(new >= 0, old >= 0) and (new < cap).all()
            stay = (old >= 0) & (old < cap)
            assert np.array_equal(new[stay], old[stay])
            went += int((old >= cap).sum())
            slots += new[new >= 0].tolist()
        assert len(set(slots)) == len(slots) == used and moved == went
        opt = env.pool.opt.view(-1, env.PR * env.E * 2)
        opt[cap:300] = 0x5A  # lent out
        sels = {x: env.select(x) for x in live if env.len[x]}
        if sels:
            env.decode(sels)
        assert bool((opt[cap:300] == 0x5A).all())
        assert env.pool.compact(300) == (0, 0)


def test_compact_order_is_lowest_page_to_lowest_hole(dhs):
    env = Env(dhs, R=4, S=1, n=64, pages=16)
    for r in range(4):
        env.admit(r, 64, resident=2.0)
    assert env.pool.release(0) == 0 and env.pool.release(2) == 0
    assert [env.state(r, 0)[2][:4].tolist() for r in (1, 3)] == [[4, 5, 6, 7], [12, 13, 14, 15]]
    assert env.pool.compact(8) == (0, 4)
    assert [env.state(r, 0)[2][:4].tolist() for r in (1, 3)] == [[4, 5, 6, 7], [0, 1, 2, 3]]
    env.decode({r: env.select(r) for r in (1, 3)})


def test_compact_limits_admission_and_refill(dhs):
    env = Env(dhs, R=3, S=1, n=64, pages=16, reserve=1)
    env.admit(0, 64, resident=2.0)
    assert env.pool.compact(6) == (0, 0)
    mask = np.ones(4, np.uint8)
    rows = torch.zeros(64, env.E, dtype=torch.int16, device="cuda")
    rc, deficit = env.pool.admit_device(1, 0, rows.data_ptr(), env.host[1, 0].data_ptr(), 64, mask)
    assert rc == dhs.DHS_EWOULDWAIT and deficit == 3
    assert env.fork(0, 1, expect=dhs.DHS_EWOULDWAIT) == 3
    assert env.fork(0, 1, [np.zeros(4)]) == 0
    assert env.pool.refill(10) == (0, 1)  # 5 usable slots
    assert env.pool.compact(4)[0] == dhs.DHS_EWOULDWAIT
    assert env.pool.capacity() == 6
    assert env.pool.compact(16) == (0, 0)
    assert env.pool.refill(10) == (0, 3)
    env.decode({r: env.select(r) for r in (0, 1)})


def test_compact_refusals(dhs):
    env = Env(dhs, pages=20)
    for cap in (-1, 21, 2 ** 40):
        assert env.pool.compact(cap)[0] == dhs.DHS_EINVAL
    assert env.pool.compact(0) == (0, 0) and env.pool.capacity() == 0
    assert env.pool.compact(20) == (0, 0)


def test_fork_and_compact_large_pages(dhs):
    """Pages beyond 16 MiB (64 KB rows)."""
    env = Env(dhs, R=3, S=1, n=1100, PR=512, T=4, B=4, E=32768, pages=6, k=2, max_rows=1104)
    env.admit(0, 1100, resident=2.0)
    env.decode({0: env.select(0)})
    env.fork(0, 1)
    env.same_step(0, 1)
    assert env.pool.release(0) == 0
    assert env.pool.compact(2) == (0, 2)
    env.decode({1: env.select(1)})
