"""The GPU tests of the int8 path once more on the debug build, in which every
plain global-memory access of a kernel checks its index against the extent of
its buffer (see test_gpu_debug_bounds.py)."""
import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.mark.gpu
def test_int8_path_under_bounds_checks():
    env = dict(os.environ, SLOPE_DEBUG_BOUNDS="1")
    cmd = [sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p", "no:cacheprovider", os.path.join(HERE, "test_gpu_q8.py")]
    res = subprocess.run(cmd, env=env, cwd=ROOT, capture_output=True, text=True, timeout=1200)
    tail = res.stdout[-4000:] + res.stderr[-2000:]
    assert res.returncode == 0, tail
    assert " passed" in res.stdout and "SLOPE_ERR_BOUNDS" not in res.stdout, tail
