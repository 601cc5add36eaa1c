"""A process whose first rotation, packing, attention over packed rows and reading
back are captured; and a prompt's chunk of many new queries over its history."""
import os
import subprocess
import sys

import pytest

from packed_layouts import LAYOUTS
from test_gpu_packed_attend import History, dhs, run  # noqa: F401

pytestmark = pytest.mark.gpu

SCRIPT = """
import torch
from packed_layouts import LAYOUTS
from test_gpu_packed_attend import Located, check_located
from hierarchical_sparse_kv_dhs_gb300 import dhs

side = torch.cuda.Stream()
with torch.cuda.stream(side):
    lay, n = LAYOUTS["%s"], 200
    env = Located(dhs, lay, seed=1)
    loc = env.rand_loc(2, 3000)
    it, t = env.item(loc)
    raw = torch.empty_like(t[0])
    turns = torch.from_numpy(dhs.rope_table(16)).cuda()
    at = torch.tensor([5, 70000], dtype=torch.int32, device="cuda")
    rot = dhs.make_rotate(raw, at, turns, out=t[0], rotary=16)
    part = lambda m: torch.empty(n, lay.kv, m, dtype=lay.type, device="cuda")
    key, wide, value = part(lay.key8), part(lay.wide) if lay.wide else None, None if lay.shared else part(lay.value)
    packed = torch.empty(n, lay.row_bytes, dtype=torch.uint8, device="cuda")
    st, keep = dhs.make_pack([dhs.pack_item(n, key, wide=wide, value=value, rows=packed)], lay.rows(dhs))
    back = part(lay.key)
    rd, keep2 = dhs.make_unpack([dhs.unpack_item(n, back, rows=packed)], lay.rows(dhs))
    att, keep3 = dhs.make_attend_packed([it], lay.rows(dhs), heads=lay.heads, scale=lay.scale)
    work = torch.empty(max(256, env.pool.attend_packed_bytes(att)), dtype=torch.uint8, device="cuda")
    att.work_dev, att.work_bytes = work.data_ptr(), work.numel()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    graph.capture_begin()
    assert env.pool.stream == side
    for rc in (env.pool.rotate(rot), env.pool.pack(st), env.pool.unpack(rd), env.pool.attend_packed(att)):
        assert rc == 0
    graph.capture_end()
    for _ in range(2):
        for x in (raw, key, wide, value):
            if x is not None:
                x.normal_(generator=env.g)
        t[1].zero_()
        graph.replay()
        check_located(env, [(loc, t)])
        assert torch.equal(back, lay.numbers(packed)[0].to(lay.type))
        assert (t[0][1, :, :16] != raw[1, :, :16]).float().mean() > 0.9 and torch.equal(t[0][..., 16:], raw[..., 16:])
    assert env.pool.status() == (0, 0)
print("captured")
"""


@pytest.mark.parametrize("name", ["latent", "grouped", "grouped_some_wide"])
def test_first_calls_are_captured(name):
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([here, os.path.dirname(here)]))
    r = subprocess.run([sys.executable, "-c", SCRIPT % name], env=env, cwd=here,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout == "captured\n", r.stdout + r.stderr


@pytest.mark.parametrize("Q", [65, 300])
@pytest.mark.parametrize("name", ["latent", "latent_100", "grouped", "grouped_f16", "odd"])
def test_a_chunk_of_queries(dhs, name, Q):  # noqa: F811
    """Many new queries: blocks of columns that end inside a query's heads, each with
    rows that only some of its columns see."""
    env = History(dhs, LAYOUTS[name], [700, Q, 3], seed=Q)
    its = env.items(Q)
    run(dhs, env.pool, env.lay, [i for i, _ in its])
    env.check(its, Q)
    assert env.pool.status() == (0, 0)
