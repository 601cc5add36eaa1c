"""Attention over packed rows whose keys and queries are far from 1, scores that are
not: what the codes, scales and queries stand for counts, not the order of the
products."""
import pytest
import torch

from packed_layouts import LAYOUTS, Layout
from test_gpu_packed_attend import Located, check_located, dhs, run  # noqa: F401

pytestmark = pytest.mark.gpu


def sized(dhs, name, keys, queries):  # noqa: F811
    """Random rows with keys 2^keys times as large, queries 2^queries times, and a
    scale that makes up for both."""
    lay = LAYOUTS[name]
    lay = Layout(lay.heads, lay.key, lay.value, lay.kv, lay.wide, lay.shared, lay.dtype)
    env = Located(dhs, lay, B=100, seed=40)
    lay.scale *= 2.0 ** -(keys + queries)
    loc = env.distinct(200)
    rows, _ = env.rows(loc)
    rows = rows[0]
    scales = rows[:, lay.off_scale:lay.off_scale + 4 * lay.scales].contiguous().view(torch.float32)
    scales[:, :lay.kv] *= 2.0 ** keys
    rows[:, lay.off_scale:lay.off_scale + 4 * lay.scales] = scales.view(torch.uint8)
    env.write(loc, rows)
    it, t = env.item(loc)
    t[0].copy_((t[0].double() * 2.0 ** queries).to(lay.type))
    run(dhs, env.pool, lay, [it])
    check_located(env, [(loc, t)])
    assert env.pool.status() == (0, 0)


@pytest.mark.parametrize("keys", [-56, 100, 112, 118])
@pytest.mark.parametrize("name", ["no_wide", "grouped", "same"])
def test_key_sizes(dhs, name, keys):  # noqa: F811
    """Key scales up to 2^116 and down to 2^-64."""
    sized(dhs, name, keys, -100 if keys > 0 else 40)


@pytest.mark.parametrize("queries", [-90, -105, -112, -118, -125])
@pytest.mark.parametrize("name", ["no_wide", "grouped", "same"])
def test_query_sizes(dhs, name, queries):  # noqa: F811
    """Queries down to bf16's subnormal ones, whose bits count as any others'."""
    sized(dhs, name, 30, queries)
