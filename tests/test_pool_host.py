"""The pool's host side without a GPU: pool.cpp linked against stand-ins for
the CUDA calls and the kernels' launchers (pool_host.cpp), one process a
scenario."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
PKG = os.path.join(os.path.dirname(HERE), "hierarchical_sparse_kv_dhs_gb300")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    if not os.path.exists(os.path.join(cuda, "cuda_runtime.h")):
        pytest.skip("no CUDA headers")
    exe = str(tmp_path_factory.mktemp("pool_host") / "pool_host")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-Wno-mismatched-new-delete", "-I", os.path.join(PKG, "csrc"),
                    "-I", os.path.join(os.path.dirname(HERE), "include"), "-I", cuda,
                    os.path.join(HERE, "pool_host.cpp"), os.path.join(PKG, "csrc", "pool.cpp"),
                    "-o", exe], check=True)
    return exe


@pytest.mark.parametrize("scenario", ["fork_of_fewer_sources", "fork_without_memory",
                                      "fork_table_limits", "calls_without_memory",
                                      "flush_behind_side_attention"])
def test_scenario(program, scenario):
    r = subprocess.run([program, scenario], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr
