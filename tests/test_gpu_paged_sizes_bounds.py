"""The bounds-checked debug build at the sizes of tests/test_gpu_paged_sizes.py:
every global access that a thread issues lies inside its tensor.  Runs
tests/paged_sizes_bounds_cases.py in a process of its own, because the package
picks its library (RF_GB300_LIB=debug) at import."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_debug_build_runs_the_larger_sizes_clean():
    env = dict(os.environ, RF_GB300_LIB="debug")
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "paged_sizes_bounds_cases.py")],
                       cwd=ROOT, env=env, stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                       text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-4000:]
    assert "every case of these sizes clean" in r.stdout
