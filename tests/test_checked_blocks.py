"""The 8-bit and gated operators' tests again under the bounds-checked build: an
index that a kernel computes outside its buffer fails the test that caused it."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
@pytest.mark.skipif(os.environ.get("SHMM_CHECKED") == "1", reason="already running under the checked build")
def test_under_the_bounds_checked_build():
    from partial_sum_reduction_gb300 import build
    build.build(checked=True)
    env = dict(os.environ, SHMM_CHECKED="1")
    files = ["test_blocks8.py", "test_scaled_matmul.py", "test_gated.py", "test_blocks_ordering.py"]
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider"] +
                       [os.path.join(ROOT, "tests", f) for f in files],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=1500)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
