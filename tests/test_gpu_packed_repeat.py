"""Attention over packed rows gives the same bits on every run: jobs whole and
split, rows of every tier, ragged histories, more jobs than blocks."""
import pytest
import torch

from packed_layouts import LAYOUTS
from test_gpu_packed_attend import History, Located, check_located, dhs, run  # noqa: F401

pytestmark = pytest.mark.gpu
TIMES = 25


def bits(ts):
    return [t.clone().view(torch.int16 if t.element_size() == 2 else torch.int32) for t in ts]


def again(dhs, env, items, outs):  # noqa: F811
    """The first run's bits against those of every later one."""
    run(dhs, env.pool, env.lay, items)
    torch.cuda.synchronize()
    first = bits(outs)
    for _ in range(TIMES):
        for t in outs:
            t.zero_()
        run(dhs, env.pool, env.lay, items)
        torch.cuda.synchronize()
        for a, b in zip(first, bits(outs)):
            assert torch.equal(a, b)
    assert env.pool.status() == (0, 0)


@pytest.mark.parametrize("name", ["latent", "latent_64_f16", "latent_128", "grouped", "grouped_f16",
                                  "no_wide_64"])
@pytest.mark.parametrize("shape", [(1, 1, 256), (8, 1, 2048), (24, 8, 1000), (3, 7, 333)])
def test_located_repeats(dhs, name, shape):  # noqa: F811
    items, Q, k = shape
    env = Located(dhs, LAYOUTS[name], B=300, seed=21)
    cases, its = [], []
    for _ in range(items):
        loc = env.rand_loc(Q, k)
        loc[torch.rand(loc.shape, generator=env.g, device="cuda") < 0.03] = 0xFFFFFFFF
        it, t = env.item(loc)
        its.append(it)
        cases.append((loc, t))
    again(dhs, env, its, [x for _, t in cases for x in t[1:3]])
    check_located(env, cases[:2])


@pytest.mark.parametrize("name", ["latent", "latent_f16", "grouped", "grouped_f16"])
def test_histories_repeat(dhs, name):  # noqa: F811
    env = History(dhs, LAYOUTS[name], [3000, 1, 777, 128, 2049], T=100, seed=22)
    its = env.items(4)
    again(dhs, env, [i for i, _ in its], [x for _, t in its for x in t[1:3]])
    env.check(its, 4)
