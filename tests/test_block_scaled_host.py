"""The block-scaled operators without a GPU: what the kernels' sources must not hold, and the host side on
stand-ins for CUDA tensors and for the CUDA runtime."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "convolution_onnx_conv_gb300", "csrc")


def source(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("name", ["k_quant.cu", "linear_dev.cuh", "tc_linear_few.cu", "tc_linear_many.cu"])
def test_no_read_only_loads_of_what_the_kernel_before_may_write(name):
    """The kernels begin while the kernel before them in the stream still runs and wait for it inside.  A
    read-only load (ld.global.nc) asks for data that nothing writes while the kernel runs, and an asm statement
    that is not volatile may be moved above the wait: neither may read x, an index, scales, offsets or biases."""
    text = source(name)
    assert not re.search(r"__ldg\b|\.nc\b|__ldcg|__ldca", text)
    assert not re.search(r"asm\s*\(\s*\"ld\.", text)
