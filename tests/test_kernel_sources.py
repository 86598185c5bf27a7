"""Rules that the kernels' sources keep, checked on the text (comments left out)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "swiglu_gated_mlp_gb300", "csrc")


def code(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


OVERLAPPING = sorted(os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu")) if "pdl_wait(" in code(p))


def test_the_fused_kernels_are_covered():
    assert {"backward_pair.cu", "fused_large_m_pair.cu", "fused_small_m.cu", "lora_shrink.cu"} <= set(OVERLAPPING)


@pytest.mark.parametrize("name", OVERLAPPING + ["ptx.cuh", "lora_lb.cuh"])
def test_no_read_only_loads_where_grids_overlap(name):
    # A read-only load asks for memory that nothing writes while the kernel is resident, and
    # may be moved ahead of the grid-dependency wait. A kernel that starts while the one
    # before it still writes its inputs may not use one, nor promise it by __restrict__.
    text = code(os.path.join(CSRC, name))
    for word in ("__ldg", "ld.global.nc", "__restrict__"):
        assert word not in text, word
