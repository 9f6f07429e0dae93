"""The tests of the 8-bit calls at their edges under the PA_DEBUG build: no block table entry behind the last one in use is
read, and no other index check fails."""
import os
import subprocess
import sys

import pytest

from paged_kv_cache_457_b200 import build_lib

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CASES = ["tests/test_gpu_fp8_row_groups.py", "tests/test_gpu_fp8_table_views.py", "tests/test_gpu_fp8_v_scales.py",
         "tests/test_gpu_fp8_hints.py", "tests/test_gpu_fp8_small_chunks.py", "tests/test_gpu_append_long.py::test_head_counts_that_do_not_divide",
         "tests/test_gpu_append_long.py::test_queries_turned_in_place"]


def test_debug_build_passes_the_edge_tests():
    lib = build_lib.build(debug=True)
    env = dict(os.environ, PA_B200_LIBRARY=lib, PA_B200_EXPECT_DEBUG="1")
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider"] + CASES
    r = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=1200)
    tail = (r.stdout + r.stderr)[-4000:]
    assert r.returncode == 0, tail
    assert " passed" in r.stdout and "failed" not in r.stdout, tail
