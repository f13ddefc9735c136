"""The debug build's index checks on the suites of the loss and tensor-list
calls' special cases, as test_gpu_zz_checked.py has them on the shard steps'."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SUITES = ["test_gpu_logits_large.py", "test_gpu_losses_reach.py", "test_gpu_preference_infinite.py",
          "test_gpu_tensors_special.py"]


def test_special_cases_under_index_checks(zs, cuda_device):
    from zero_partitioned_mixed_partition_gb300 import build
    build.build(checked=True)
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
           *[os.path.join(ROOT, "tests", f) for f in SUITES]]
    r = subprocess.run(cmd, cwd=ROOT, env=dict(os.environ, ZS_CHECKED="1"), capture_output=True, text=True, timeout=900)
    tail = "\n".join((r.stdout + r.stderr).strip().splitlines()[-15:])
    assert r.returncode == 0 and " passed" in tail and "failed" not in tail, tail
