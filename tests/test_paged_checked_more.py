"""More of the cache in pages against the checked build, in a child process: padded and large ragged batches, workspaces of the planned
size, lengths that change under a call."""
import os
import subprocess
import sys

import pytest

from head_attention_forward_fmha_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_edges_pass_with_index_checks():
    env = dict(os.environ, FMHA_GB300_LIB=build.build(checked=True))
    files = ["tests/test_paged_edges.py", "tests/test_paged_workspace.py", "tests/test_paged_changing_lengths.py", "tests/test_kv4_changing_lengths.py"]
    r = subprocess.run([sys.executable, "-m", "pytest", *files, "-m", "gpu", "-x", "-q", "-p", "no:cacheprovider", "-k",
                        "search or more_tokens or planned or change"], env=env, cwd=ROOT, capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, "\n".join((r.stdout + r.stderr).splitlines()[-30:])
