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


@pytest.mark.parametrize("name", [f for f in EARLY if "tmem_alloc(" in open(os.path.join(CSRC, f)).read()])
def test_dependents_are_launched_once_tensor_memory_is_held(name):
    """A kernel launched early waits for the one in front before it gives anything back. If it could take tensor memory
    that the one in front has yet to take, both would wait for good: the warp that takes it is the one that lets the
    next launch in, after that."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    signals = [m.start() for m in re.finditer(r"launch_dependents\(\)", text)]
    takes = [m.start() for m in re.finditer(r"tmem_alloc\(", text)]
    assert len(signals) == len(takes) == 1
    assert re.fullmatch(r"tmem_alloc\([^;]*;\s*umma::tmem_relinquish\(\);\s*pipe::", text[takes[0]:signals[0]])
