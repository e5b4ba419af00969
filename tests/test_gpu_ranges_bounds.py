"""The GPU tests of the norm's range, the product's scales and the pair kernels'
codes once more on the debug build (see test_gpu_debug_bounds.py)."""
import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
FILES = ["test_gpu_norm_range.py", "test_gpu_q8_scales.py", "test_gpu_q8_slices.py", "test_pair_ordering.py"]


@pytest.mark.gpu
def test_under_bounds_checks():
    env = dict(os.environ, SLOPE_DEBUG_BOUNDS="1")
    cmd = [sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p", "no:cacheprovider"] + [os.path.join(HERE, f) for f in FILES]
    res = subprocess.run(cmd, env=env, cwd=ROOT, capture_output=True, text=True, timeout=900)
    tail = res.stdout[-4000:] + res.stderr[-2000:]
    assert res.returncode == 0, tail
    assert " passed" in res.stdout and "SLOPE_ERR_BOUNDS" not in res.stdout, tail
