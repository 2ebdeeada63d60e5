"""Beam search and adapters in the bounds-checking build (see tests/test_bounds_check_gpu.py):
every address their kernels compute passes its check."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_beam_and_adapter_kernels_pass_their_bounds_checks():
    from vocabulary_cross_entropy_gb300 import build
    env = dict(os.environ, VCE_LIBRARY=build.build_bounds_check())
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "beam_bounds_cases.py")], env=env,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "beam bounds cases ok" in r.stdout
