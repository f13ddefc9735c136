"""Exhaustive GPU checks of the packed square root, reciprocal and divisions of
the AdamW step over a list of tensors, by the program
tests/gpu_tensors_math_check.cu (compiled here for sm_103a): bit for bit the
correctly rounded scalar operations, over the ranges that the step uses them in."""
import os
import shutil
import subprocess

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_tensors_math_exhaustive(cuda_device, tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    exe = str(tmp_path / "tensors_math_check")
    csrc = os.path.join(ROOT, "zero_partitioned_mixed_partition_gb300", "csrc")
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-std=c++17", "-I", csrc,
                    os.path.join(ROOT, "tests", "gpu_tensors_math_check.cu"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    print(r.stdout)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.strip().endswith("all equal")
    assert r.stdout.count(": 0 mismatches") == 2 + 40 + 10
