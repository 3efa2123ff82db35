"""The int8 layers' many-rows kernel, and every other form, under the bounds-checking build (CONVF_DEBUG_BOUNDS): each row and
column of y that is stored by index arithmetic is checked against y; the cases have to match with status CONVF_OK."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_many_rows_under_the_bounds_checking_build():
    env = dict(os.environ, CONVF_DEBUG_BOUNDS="1")
    subprocess.run([sys.executable, "-c", "from convolution_onnx_conv_gb300 import _build; "
                    "_build.build(debug_bounds=True)"], cwd=ROOT, env=env, check=True)
    res = subprocess.run([sys.executable, "-m", "pytest", os.path.join("tests", "test_gpu_linear_int8_many.py"), "-m", "gpu", "-q", "-x",
                          "-p", "no:cacheprovider", "-k", "every_way_out or test_experts or short_reduction or zeros_keep"],
                         cwd=ROOT, env=env, capture_output=True, text=True)
    assert res.returncode == 0 and " passed" in res.stdout, (res.stdout + res.stderr)[-3000:]
