"""Rules of the kernels' sources that no run can show broken: the GPU may order things kindly for years."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "precision_integer_gemm_gb300", "csrc")


def code_of(name):
    """A source without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("name", ["pack_fp4.cu", "moe.cu", "gemm_fp4_kernel.cuh", "gemm_fp4.cuh"])
def test_kernels_set_up_early_make_no_read_only_loads(name):
    # a read-only load, or one through a const restrict pointer, promises that nobody writes the memory during the
    # kernel's life; that of a kernel launched ahead of the end of the one before it begins while that one writes
    code = code_of(name)
    assert "griddepcontrol.wait" in code or "overlap" in code or name == "gemm_fp4.cuh"
    for word in ("__ldg", "__ldcg", "__ldcs", "__restrict__", "ld.global.nc"):
        assert word not in code, word
