"""Rules that the sources of the operators around the attention keep, checked
without a GPU."""

import os
import re

import pytest

from block_sparse_long_bwd_b200 import binding as bb

CSRC = os.path.join(os.path.dirname(bb.LIB_PATH), "csrc")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"/\*.*?\*/", "", re.sub(r"//[^\n]*", "", text), flags=re.S)


@pytest.mark.parametrize("name", ["layer.cuh", "out_dropout.cu", "qk_rope.cu", "linear_ce.cu"])
def test_chained_kernels_load_coherently(name):
    """A kernel that is launched while the one in front still runs reads what
    that one writes.  The non-coherent path (__ldg, ld.global.nc, what const
    __restrict__ pointers allow) is for memory that nothing writes during the
    kernel's whole life, the time before its wait included."""
    code = _code(name)
    assert not re.search(r"__ldg|ld\.global\.nc|__restrict__", code)


@pytest.mark.parametrize("name", ["out_dropout.cu", "qk_rope.cu", "linear_ce.cu"])
def test_every_chained_kernel_waits_once(name):
    """Each kernel waits for the launches in front, on every path, exactly once
    and right after it lets the next one begin."""
    code = _code(name)
    kernels = len(re.findall(r"__global__ void", code))
    pairs = re.findall(r"grid_launch_dependents\(\);\s*(?:sm100::)?grid_wait\(\);", code)
    assert kernels == len(pairs) == len(re.findall(r"grid_wait\(\)", code))
