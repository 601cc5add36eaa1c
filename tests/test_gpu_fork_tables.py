"""Forks and compactions larger than the tables that travel with a launch."""
import pytest

from test_gpu_fork import Env, dhs  # noqa: F401

pytestmark = pytest.mark.gpu


def test_fork_of_more_pages_than_a_launch_lists(dhs):  # noqa: F811
    n = 16 * 7000
    env = Env(dhs, R=2, S=1, n=n, pages=14100, k=200, B=500)
    env.admit(0, n, resident=1.0)
    env.decode({0: env.select(0)})
    env.fork(0, 1)
    env.same_state(0, 1)
    for _ in range(3):
        env.append([0, 1], 2)
        env.same_step(0, 1)


@pytest.mark.parametrize("n", [1000, 4000])
def test_compaction_of_many_runs(dhs, n):  # noqa: F811
    """Pages whose map entries have gaps move in as many runs as there are gaps."""
    env = Env(dhs, R=3, S=2, n=n, pages=2 * 3 * n // 16)
    for r in range(3):
        env.admit(r, n, resident=0.6)
    assert env.pool.release(0) == 0
    before = env.pool.used()
    rc, moved = env.pool.compact(before)
    assert rc == 0 and moved > 32 and env.pool.capacity() == before == env.pool.used()
    for _ in range(3):
        env.append([1, 2], 1)
        env.decode({1: env.select(1), 2: env.select(2)})
