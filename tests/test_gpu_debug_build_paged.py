"""The packed, tree and paged calls in libgqa_debug.so (device-side index checks): the same tests pass,
and every one of them reads the status word, so a check that fires fails it."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_packed_tree_and_paged_calls_pass_with_index_checks():
    files = ["tests/test_gpu_packed.py", "tests/test_gpu_tree.py", "tests/test_gpu_pages.py",
             "tests/test_gpu_serving_run.py", "tests/test_gpu_paged_limits.py"]
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "gpu", *files],
                       cwd=ROOT, env=dict(os.environ, GQA_LIB="debug"), capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
