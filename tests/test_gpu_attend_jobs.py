"""Attention: how a launch's jobs are dealt to the blocks - whole jobs in
waves, a split rest, fewer blocks than SMs, more segments a block than are
found ahead, jobs cut into more parts than a warp has lanes."""
import pytest
import torch

from test_gpu_attend import LAYOUTS, History, Located, check_located, dhs, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["latent", "latent_64", "grouped", "odd"])
@pytest.mark.parametrize("queries,k", [(160, 300), (304, 140), (100, 128), (170, 100), (700, 60),
                                       (8, 2000), (20, 1200)])
def test_equal_jobs(dhs, name, queries, k):  # noqa: F811
    env = Located(dhs, LAYOUTS[name], seed=queries)
    cases, items = [], []
    while queries:
        Q = min(8, queries)
        loc = env.rand_loc(Q, k)
        it, t = env.item(loc)
        items.append(it)
        cases.append((loc, t))
        queries -= Q
    run(dhs, env.pool, env.lay, items)
    check_located(env, cases)
    assert env.pool.status() == (0, 0)


@pytest.mark.parametrize("name", ["latent_128", "grouped_f16"])
def test_short_jobs_between_empty_and_long_ones(dhs, name):  # noqa: F811
    env = Located(dhs, LAYOUTS[name], seed=3)
    cases, items = [], []
    for i in range(60):
        loc = env.rand_loc(1 + i % 3, (0, 1, 700, 0, 128, 5, 0, 0, 0, 129)[i % 10])
        it, t = env.item(loc)
        items.append(it)
        cases.append((loc, t))
    run(dhs, env.pool, env.lay, items)
    check_located(env, cases)


@pytest.mark.parametrize("name", ["latent", "latent_100", "grouped"])
@pytest.mark.parametrize("k", [4300, 21000])
def test_a_job_in_many_parts(dhs, name, k):  # noqa: F811
    env = Located(dhs, LAYOUTS[name], seed=k)
    loc = env.rand_loc(2, k)
    loc[1, 128:k - 128] = 0xFFFFFFFF  # parts without a row between parts with some
    it, t = env.item(loc)
    run(dhs, env.pool, env.lay, [it])
    check_located(env, [(loc, t)])


@pytest.mark.parametrize("Q", [1, 5])
def test_equal_histories(dhs, Q):  # noqa: F811
    env = History(dhs, LAYOUTS["grouped"], [600] * 24, seed=Q)
    its = env.items(Q)
    run(dhs, env.pool, env.lay, [i[0] for i in its])
    env.check(its, Q)
    torch.cuda.synchronize()
    assert env.pool.status() == (0, 0)
