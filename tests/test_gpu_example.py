"""examples/branch_decode.py: attention, forks and compaction together."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("steps,rows", [(4, 2000), (3, 777)])
def test_branch_decode(steps, rows):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "branch_decode.py")
    spec = importlib.util.spec_from_file_location("branch_decode", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    done = mod.main(["--steps", str(steps), "--rows", str(rows), "--check"])
    assert done["requests"] == 2 and done["capacity"] == done["pages"]
    # weights and outputs are rounded to bf16 once each, by at most 2^-9 of
    # their own size and independently: sqrt(2) 2^-9 together over a row
    assert done["error"] <= 2 ** -8
