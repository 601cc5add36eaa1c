"""examples/packed_decode.py: rotation, packing, appending, reading back and
attention in 8 bits together, with resolves, a fork and a compaction."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("steps,rows", [(4, 2000), (3, 777), (0, 512)])
def test_packed_decode(steps, rows):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "packed_decode.py")
    spec = importlib.util.spec_from_file_location("packed_decode", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    done = mod.main(["--steps", str(steps), "--rows", str(rows), "--check"])
    assert done["requests"] == (2 if steps else 3)
    if steps:
        assert done["capacity"] == done["pages"]
    # the output is rounded by at most 2^-8 of itself, a weight by 2^-9 + 2^-11
    # (three pieces of a number rounded to f16); the float sums add less than
    # 2^-13 of the whole
    assert done["error"] <= 2 ** -8 + 2 ** -9 + 2 ** -11 + 2 ** -13
    # a code is off by at most 2^-4 of its element, or by 2^-10 of the scale, of
    # which the largest element has 224 or more: together 512 such elements have
    # sqrt(512) 2^-10 / 224 < 2^-13 of the row's length
    assert done["held"] <= 2 ** -4 + 2 ** -13
