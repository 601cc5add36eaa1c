"""Attention captured into a CUDA graph, also as the first attention of a process."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

SCRIPT = """
import torch
from test_gpu_attend import LAYOUTS, History, Located, check_located
from hierarchical_sparse_kv_dhs_gb300 import dhs

side = torch.cuda.Stream()
with torch.cuda.stream(side):
    lay = LAYOUTS["%(name)s"]
    env = Located(dhs, lay, seed=1)
    loc = env.rand_loc(2, 3000)
    it, t = env.item(loc)
    st, keep = dhs.make_attend([it], **lay.args())
    work = torch.empty(max(256, env.pool.attend_bytes(st)), dtype=torch.uint8, device="cuda")
    st.work_dev, st.work_bytes = work.data_ptr(), work.numel()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    graph.capture_begin()
    assert env.pool.stream == side and env.pool.attend(st) == 0
    graph.capture_end()
    for seed in (1, 2):  # other queries, the same graph
        t[0].normal_(generator=env.g)
        t[1].zero_()
        graph.replay()
        check_located(env, [(loc, t)])
    assert env.pool.status() == (0, 0)
print("captured")
"""


@pytest.mark.parametrize("name", ["latent", "latent_128", "grouped"])
def test_first_attention_is_captured(name):
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([here, os.path.dirname(here)]))
    r = subprocess.run([sys.executable, "-c", SCRIPT % dict(name=name)], env=env, cwd=here,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout == "captured\n", r.stdout + r.stderr
