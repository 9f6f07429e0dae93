"""The rotating and 8-bit calls under the PA_DEBUG build: every index the kernels derive is checked on the device before
use, and no check may fail.  As for the other kernels, the tests run in a child process that loads
libpa_b200_debug.so; the fixture of conftest.py looks at the status word after every one."""
import os
import subprocess
import sys

import pytest

from paged_kv_cache_457_b200 import build_lib

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CASES = ["tests/test_gpu_append.py", "tests/test_gpu_fp8_decode.py", "tests/test_gpu_fp8_prefill.py",
         "tests/test_gpu_fp8_serving.py"]


def test_debug_build_passes_the_8_bit_tests():
    lib = build_lib.build(debug=True)
    env = dict(os.environ, PA_B200_LIBRARY=lib, PA_B200_EXPECT_DEBUG="1")
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider"] + CASES
    r = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=1200)
    tail = (r.stdout + r.stderr)[-4000:]
    assert r.returncode == 0, tail
    assert " passed" in r.stdout and "failed" not in r.stdout, tail
