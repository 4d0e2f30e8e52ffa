"""The training and adapter operators under the bounds-checked build
(libshmm_checked.so): their GPU suites run again in a child process with
SHMM_CHECKED=1, where an index outside its buffer skips the access and leaves
SHMM_ERR_BOUNDS in the device status word.  The suites' last word here is that
status, whatever calls their own tests check it after."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

RUN = """
import sys, pytest
code = pytest.main(["-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", sys.argv[1]])
import partial_sum_reduction_gb300 as s
s.shmm_sync_status()
sys.exit(int(code))
"""


@pytest.mark.parametrize("suite", ["test_layernorm_training.py", "test_adapters.py"])
def test_suite_passes_under_bounds_checks(suite):
    from partial_sum_reduction_gb300 import build
    build.build(checked=True)
    env = dict(os.environ, SHMM_CHECKED="1")
    r = subprocess.run([sys.executable, "-c", RUN, os.path.join("tests", suite)], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-6000:] + r.stderr[-3000:]
    assert " passed" in r.stdout and "failed" not in r.stdout, r.stdout[-3000:]
