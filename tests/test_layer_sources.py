"""What the layer's kernels are written with (CPU: their sources are read)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "conditional_draft_tree_lm_gb300", "csrc")


def code(path):
    """A source file without its comments."""
    with open(path) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def test_kernels_that_begin_beside_the_one_before_them_read_by_ordinary_loads():
    """Read-only loads are for memory that nobody writes while the kernel runs; loads by intrinsics need not stay behind the wait."""
    behind = [p for p in glob.glob(os.path.join(CSRC, "*.cu")) if "launch_behind(" in code(p)]
    assert {os.path.basename(p) for p in behind} >= {"linear.cu", "linear_token.cu", "linear_wide.cu", "rotate.cu", "logprobs.cu"}
    for path in behind + [os.path.join(CSRC, "linear.cuh"), os.path.join(CSRC, "cluster.cuh")]:
        assert not re.search(r"__ld[gc]\w*\b|\.global(\.\w+)*\.nc\b|__restrict__", code(path)), os.path.basename(path)
