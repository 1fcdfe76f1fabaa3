"""Kernels that are launched before the one in front of them has ended read
nothing through the read-only path: it takes for granted that the data does
not change while the kernel runs, and the kernel in front may still write it
(the lengths or the bias that a kernel of the same stream makes)."""
import os
import re

import pytest

import nvfp4_block_scaled_12_b200 as F

CSRC = os.path.join(os.path.dirname(F.__file__), "csrc")


def _code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def _launched_early():
    return [n for n in sorted(os.listdir(CSRC)) if n.endswith(".cu") and "wait_for_previous_kernel()" in _code(n)]


def test_the_files_with_kernels_launched_early():
    assert _launched_early() == ["attention.cu", "gemm.cu", "quantize.cu", "rope.cu"]


@pytest.mark.parametrize("name", ["attention.cu", "quantize.cu", "rope.cu"])
def test_no_read_only_loads(name):
    assert not re.findall(r"__ldg|ld\.global\.nc|__restrict__ const", _code(name))


def test_the_gemm_reads_its_bias_by_the_launch():
    code = _code("gemm.cu")
    assert "p.bias" in code and not re.findall(r"__ldg\([^;]*p\.bias", code)
    # what else it reads that way belongs to variants that are not launched early
    for use in re.findall(r"__ldg\(([^;]*)\)", code):
        assert use == "p" or "row_scale" in use or "col_scale" in use, use
