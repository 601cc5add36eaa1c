"""examples/branch_decode.py over hundreds of steps, and over one."""
import pytest

import test_gpu_example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("steps,rows", [(300, 512), (1, 512)])
def test_other_lengths(steps, rows):
    test_gpu_example.test_branch_decode(steps, rows)
