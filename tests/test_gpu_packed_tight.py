"""Shared rows whose tile takes five slots of codes and one of wide elements: there is
no room for two tiles at any width, and a tile's loads, scores, weights and sums
follow each other."""
import pytest
import torch

from packed_layouts import Layout
from test_gpu_packed_attend import History, Located, check_located, dhs, run  # noqa: F401

pytestmark = pytest.mark.gpu

TIGHT = {
    "wide_16": Layout(16, 576, 512, wide=16, shared=True),
    "wide_32": Layout(40, 576, 512, wide=32, shared=True),
    "wide_48": Layout(64, 576, 512, wide=48, shared=True),
    "wide_48_f16": Layout(24, 576, 512, wide=48, shared=True, dtype="f16"),
    "wide_16_f16": Layout(128, 576, 512, wide=16, shared=True, dtype="f16"),
    "all_coded": Layout(17, 576, 512, shared=True),
    "all_coded_f16": Layout(33, 576, 512, shared=True, dtype="f16"),
    "two_heads": Layout(34, 576, 400, kv=2, wide=48, shared=True),
}


@pytest.mark.parametrize("k", [0, 1, 127, 129, 300, 2500])
@pytest.mark.parametrize("name", sorted(TIGHT))
def test_located(dhs, name, k):  # noqa: F811
    env = Located(dhs, TIGHT[name], seed=k)
    cases, items = [], []
    for Q in (1, 3):
        loc = env.rand_loc(Q, k)
        if k > 2:
            loc[0, 1: k // 2] = 0xFFFFFFFF
        it, t = env.item(loc)
        items.append(it)
        cases.append((loc, t))
    env.poison(torch.cat([c[0].reshape(-1) for c in cases]))
    run(dhs, env.pool, env.lay, items)
    check_located(env, cases)
    assert env.pool.status() == (0, 0)


@pytest.mark.parametrize("name", ["wide_48", "wide_16_f16", "two_heads"])
def test_many_jobs(dhs, name):  # noqa: F811
    """Several whole jobs a block, one after the other, and what is left split."""
    env = Located(dhs, TIGHT[name], seed=1)
    cases, its = [], []
    for _ in range(50):
        loc = env.rand_loc(8, 290)
        it, t = env.item(loc)
        its.append(it)
        cases.append((loc, t))
    run(dhs, env.pool, env.lay, its)
    check_located(env, cases[::13])
    assert env.pool.status() == (0, 0)


@pytest.mark.parametrize("Q", [1, 4])
@pytest.mark.parametrize("name", sorted(TIGHT))
def test_history(dhs, name, Q):  # noqa: F811
    env = History(dhs, TIGHT[name], [0, 1, 17, 128, 500, 3000], seed=Q)
    its = env.items(Q)
    run(dhs, env.pool, env.lay, [i for i, _ in its])
    env.check(its, Q)
    assert env.pool.status() == (0, 0)
