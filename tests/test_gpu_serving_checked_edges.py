"""The edge cases of the rotary, cache and single-token calls again, against the
bounds-checked build of the library (ULYSSES_CHECKED=1 in a child process)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FILES = ["tests/test_gpu_checked_variant.py", "tests/test_gpu_serving_edges.py", "tests/test_gpu_serving_inputs.py",
         "tests/test_gpu_serving_calls.py", "tests/test_gpu_multicast.py"]


def test_edges_under_the_checked_build():
    from long_context_sequence_seq_gb300 import build as B
    B.build(checked=True)
    env = {**os.environ, "ULYSSES_CHECKED": "1"}
    r = subprocess.run([sys.executable, "-m", "pytest", *FILES, "-m", "gpu", "-q", "-x", "-p", "no:cacheprovider"], cwd=ROOT,
                       env=env, capture_output=True, text=True, timeout=1200)
    tail = "\n".join((r.stdout + r.stderr).splitlines()[-30:])
    assert r.returncode == 0, tail
    assert " passed" in tail and "failed" not in tail, tail
