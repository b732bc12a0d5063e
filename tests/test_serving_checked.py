"""The serving operators' GPU tests against the checked build (every computed index tested
before its access), in a child process; tests/conftest.py reads the status word after each."""
import os
import subprocess
import sys

import pytest

from head_attention_forward_fmha_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_serving_suite_passes_with_index_checks():
    env = dict(os.environ, FMHA_GB300_LIB=build.build(checked=True))
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_serving_ops.py", "-m", "gpu", "-x", "-q", "-p", "no:cacheprovider"],
                       env=env, cwd=ROOT, capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, "\n".join((r.stdout + r.stderr).splitlines()[-30:])


@pytest.mark.gpu
def test_serving_edges_pass_with_index_checks():
    env = dict(os.environ, FMHA_GB300_LIB=build.build(checked=True))
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_serving_edges.py", "-m", "gpu", "-x", "-q", "-p", "no:cacheprovider"],
                       env=env, cwd=ROOT, capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, "\n".join((r.stdout + r.stderr).splitlines()[-30:])
