"""Forks whose page count is at, or one beside, a size of the tables of page
slots that travel with the launch (512 and 6656)."""
import pytest

from test_gpu_fork import Env, dhs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sources,pages", [(1, 511), (1, 512), (1, 513), (1, 6655), (1, 6656),
                                           (1, 6657), (4, 512), (4, 6656), (13, 6656)])
def test_fork_at_a_table_limit(dhs, sources, pages):  # noqa: F811
    n = 16 * (pages // sources)
    env = Env(dhs, R=2, S=sources, n=n, pages=2 * pages, k=64, B=200)
    env.admit(0, n, resident=2.0)
    env.decode({0: env.select(0)})
    env.fork(0, 1)
    env.same_state(0, 1)
    for _ in range(2):
        env.append([0, 1], 2)
        env.same_step(0, 1)
