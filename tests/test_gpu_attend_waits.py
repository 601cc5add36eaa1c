"""Attention whose barrier waits run out (DHS_OPT_ATTEND_POLLS): the launch
ends, says so, touches nothing but its outputs, and leaves the pool usable."""
import pytest
import torch

from test_gpu_attend import LAYOUTS, History, Located, check_located, dhs  # noqa: F401

pytestmark = pytest.mark.gpu
GUARD = 64


def attempt(dhs, pool, lay, items):  # noqa: F811
    """One call with guards around the workspace; returns the pool's status."""
    st, keep = dhs.make_attend(items, **lay.args())
    need = pool.attend_bytes(st)
    work = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    st.work_dev, st.work_bytes = work.data_ptr(), need
    if need == 0:
        st.work_dev = None
    assert pool.attend(st) == 0
    status = pool.status()
    assert bool((work[need:] == 0xA5).all())
    return status


def guarded(it, t, lay):
    """The item's outputs moved into the middle of larger buffers."""
    q, out, lse = t[:3]
    o = torch.full((out.numel() + 2 * GUARD,), 7.0, dtype=out.dtype, device="cuda")
    z = torch.full((lse.numel() + 2 * GUARD,), 7.0, device="cuda")
    it.out_dev, it.lse_dev = o[GUARD:].data_ptr(), z[GUARD:].data_ptr()
    inner = o[GUARD:-GUARD].view_as(out), z[GUARD:-GUARD].view_as(lse)
    return (q, *inner, *t[3:]), (o, z)


def untouched(guards):
    for o, z in guards:
        for x in (o, z):
            assert bool((x[:GUARD] == 7.0).all()) and bool((x[-GUARD:] == 7.0).all())


def polled(dhs, pool, polls, call, check):  # noqa: F811
    late = (dhs.DHS_ETIMEDOUT, dhs.DHS_STATUS_ETIMEDOUT)
    pool.set_option(dhs.DHS_OPT_ATTEND_POLLS, polls)
    for _ in range(3):
        status = call()
        assert status == late if polls == 0 else status in (late, (0, 0))
        if status == (0, 0):
            check()
    pool.set_option(dhs.DHS_OPT_ATTEND_POLLS, -1)
    assert call() == (0, 0)
    check()


@pytest.mark.parametrize("polls", [0, 1, 2, 7])
@pytest.mark.parametrize("name", ["latent", "latent_128", "grouped", "odd", "largest"])
def test_located(dhs, name, polls):  # noqa: F811
    """Split jobs, and more segments a block than are found ahead."""
    env = Located(dhs, LAYOUTS[name], seed=polls)
    cases, items, guards = [], [], []
    for Q, k in [(1, 2500)] + [(8, 130)] * 30 + [(8, 0)] * 40:
        loc = env.rand_loc(Q, k)
        it, t = env.item(loc)
        t, g = guarded(it, t, env.lay)
        items.append(it)
        cases.append((loc, t))
        guards.append(g)
    polled(dhs, env.pool, polls, lambda: attempt(dhs, env.pool, env.lay, items),
           lambda: check_located(env, cases))
    untouched(guards)


@pytest.mark.parametrize("polls", [0, 1, 2, 7])
@pytest.mark.parametrize("name", ["latent", "grouped"])
def test_histories(dhs, name, polls):  # noqa: F811
    """Rows on the host too, and rows whose values are not finite where only
    some queries see them."""
    env = History(dhs, LAYOUTS[name], [0, 5, 300, 2000, 5000], seed=polls)
    its, guards = [], []
    for it, t in env.items(5):
        t, g = guarded(it, t, env.lay)
        its.append((it, t))
        guards.append(g)
    call = lambda: attempt(dhs, env.pool, env.lay, [it for it, _ in its])  # noqa: E731
    polled(dhs, env.pool, polls, call, lambda: env.check(its, 5))
    # the same with the ring's rows damaged: the path for such rows
    env.pool.tail.fill_(0xFF)  # NaN
    env.pool.set_option(dhs.DHS_OPT_ATTEND_POLLS, polls)
    for _ in range(3):
        assert call()[0] in (0, dhs.DHS_ETIMEDOUT)
    untouched(guards)


def test_option(dhs):  # noqa: F811
    pool = Located(dhs, LAYOUTS["smallest"]).pool
    key = dhs.DHS_OPT_ATTEND_POLLS
    assert pool.get_option(key) == 1 << 22
    for v in (0, 5, 1 << 22, -1):
        pool.set_option(key, v)
        assert pool.get_option(key) == (v if v >= 0 else 1 << 22)
    for v in (-2, (1 << 22) + 1):
        assert dhs.lib.dhs_set_option(pool.h, key, v) == dhs.DHS_EINVAL
    assert pool.get_option(key) == 1 << 22
