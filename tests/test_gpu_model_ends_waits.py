"""The head's waits under the debug build, whose limit can be set, in a process of its
own; and its index checks on the suites of the head, norm and embedding calls."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.parametrize("suites", [["model_ends_waits_under_debug_build.py"],
                                    ["test_gpu_head.py", "test_gpu_norm.py", "test_gpu_embed.py", "test_gpu_model_ends.py"]])
def test_under_the_debug_build(zs, cuda_device, suites):
    from zero_partitioned_mixed_partition_gb300 import build
    build.build(checked=True)
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", *[os.path.join(HERE, f) for f in suites]]
    r = subprocess.run(cmd, cwd=os.path.dirname(HERE), env=dict(os.environ, ZS_CHECKED="1"), capture_output=True, text=True, timeout=900)
    tail = "\n".join((r.stdout + r.stderr).strip().splitlines()[-15:])
    assert r.returncode == 0 and " passed" in tail and "failed" not in tail, tail
