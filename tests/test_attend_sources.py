"""What the attention kernels' sources have to keep where no run can show that
it is missing: an arrival of one lane for its warp releases only what that lane
has ordered behind itself, so that the warp meets (__syncwarp) right before."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "hierarchical_sparse_kv_dhs_gb300", "csrc")
GUARD = re.compile(r"if \((?:lane == 0|\(tid & 31\) == 0)\)")


def lines_of(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    return [x.strip() for x in text.splitlines() if x.strip()]


@pytest.mark.parametrize("name", ["attend.cu", "attend_core.cuh", "attend_packed.cu"])
def test_a_warp_meets_before_one_lane_arrives(name):
    lines, arrivals = lines_of(name), 0
    for i, line in enumerate(lines):
        if not GUARD.match(line):
            continue
        body = line if ";" in line else " ".join(lines[i:i + 4])
        if "bar_arrive" not in body:
            continue
        arrivals += 1
        assert lines[i - 1] == "__syncwarp();", "%s: %s" % (name, body)
    assert arrivals >= 2


def test_a_rotation_reads_as_what_it_may_write():
    """x and y of a rotation may be one tensor: x is not read through the read-only
    path, which is for memory that the kernel does not write."""
    with open(os.path.join(CSRC, "packed_rows.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    kernel = text[text.index("rotate_kernel(const"):text.index("struct PackParams")]
    reads = re.findall(r"\b(\w+(?:<\w+>)?)\(x\b", kernel)
    assert reads and set(reads) == {"raw8<false>"}
    assert set(re.findall(r"__ldg\(([\w.]+)", kernel)) == {"r.turns", "P.position"}
    body = text[text.index("uint4 raw8("):]
    body = body[:body.index("\n}")]
    assert re.search(r"if \(CONST[^\n]*__ldg", body) and body.count("__ldg") == 1
