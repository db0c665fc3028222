"""What the loss head's kernels may wait for, read from their sources.

A wait without a limit that can fail to end hangs a GPU, so this is checked here and not there: no block waits for
another one (no clusters of blocks, no pairs of SMs on one product), and no wait for a barrier in shared memory stands
outside the functions that give up after the limit.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gradient_sync_plan_gb300", "csrc")
SOURCES = ["loss_gemm.cu", "loss_rows.cu", "loss_small.cu", "loss_api.cpp", "loss_internal.h"]


def _code(name):
    """A source without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", SOURCES)
@pytest.mark.parametrize("word", ["cta_group::2", "barrier.cluster", "mapa", "ClusterDimension", "grid.sync", "multicast"])
def test_no_block_waits_for_another(name, word):
    assert word not in _code(name)


def test_waits_for_barriers_have_a_limit():
    code = _code("loss_gemm.cu")
    # a wait's instruction stands in bar_try alone, and bar_try in the two functions that look at the clock
    assert len(re.findall(r"mbarrier\.try_wait", code)) == 1
    for body in re.split(r"\n(?=__device__|template)", code):
        if re.search(r"bar_try\(", body) and "bool bar_try(" not in body:
            assert "g.limit_ns" in body and "now_ns()" in body, body[:200]
    # and where a block asks without waiting, it does not do so in a loop of its own
    assert not re.search(r"while\s*\([^)]*bar_test", code)
