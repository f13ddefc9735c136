"""What a call of the logits kernels does when a wait of theirs runs out.  The
debug build can make them give up after a few tries, or at once, although nothing
is wrong: a row's outputs are then the usual bits or NaN throughout, never
something else, nothing outside the rows is written, and the next call is
undisturbed.  (Every wait is bounded and every address comes from what a met wait
has brought, so these calls end.)"""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_waits_that_run_out(zs, cuda_device):
    from zero_partitioned_mixed_partition_gb300 import build
    build.build(checked=True)
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
           os.path.join(ROOT, "tests", "waits_under_debug_build.py")]
    r = subprocess.run(cmd, cwd=ROOT, env=dict(os.environ, ZS_CHECKED="1"), capture_output=True, text=True, timeout=600)
    tail = "\n".join((r.stdout + r.stderr).strip().splitlines()[-15:])
    assert r.returncode == 0 and " passed" in tail and "skipped" not in tail, tail
