"""A rule of the kernels' sources that no run shows: what is launched early reads global memory by plain loads."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bitplane_mixed_precision_b200", "csrc")
EARLY = [f for f in sorted(os.listdir(CSRC)) if f.endswith(".cu") and "launch_early(" in open(os.path.join(CSRC, f)).read()]


def test_some_kernels_are_launched_early():
    assert {"group.cu", "grouped.cu", "norm_q8.cu"} <= set(EARLY)


@pytest.mark.parametrize("name", EARLY)
def test_kernels_that_are_launched_early_promise_nothing_read_only(name):
    """While such a kernel is resident the launch in front of it may still write its inputs: a read-only load (asked
    for, or chosen by the compiler for a pointer that is const and restrict) could return what was there before."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    assert "__ldg(" not in text and "ld.global.nc" not in text
    assert not re.search(r"const\s+\w+\s*\*\s*__restrict__", text)
