"""The block-scaled FP8 suites again, against the bounds-checked debug build of the library (as test_gpu_debug_bounds does
for the other kernels): after every test the build must have checked and counted no index outside its buffer."""
import os
import subprocess
import sys

import pytest

from tensor_transformer_mlp_tp_gb300 import build

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SUITES = ["tests/test_gpu_block_fp8.py", "tests/test_gpu_norm_backward_ring.py", "tests/test_gpu_block_fp8_calls.py"]


def test_block_scaled_suites_under_bounds_checks():
    lib = build.build(debug_bounds=True)
    env = dict(os.environ, TPMLP_LIBRARY=lib, TPMLP_EXPECT_BOUNDS_CHECKED="1")
    r = subprocess.run([sys.executable, "-m", "pytest", *SUITES, "-m", "gpu", "-q", "-x", "-p", "no:cacheprovider"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=1800)
    tail = "\n".join((r.stdout + r.stderr).strip().splitlines()[-25:])
    assert r.returncode == 0, tail
    assert " passed" in tail and "failed" not in tail, tail
