"""The fine-tuning example learns what its losses ask for, and the debug build's
index checks pass on the loss and tensor-list suites."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


def test_policy_steps_raise_the_rewarded_tokens(zs, cuda_device):
    import finetune_step
    totals, logp, ref, label, ctrl = finetune_step.run("policy", steps=24)
    assert ctrl["step"] == 24 and ctrl["skipped"] == 0
    good, bad = (label >= 0) & (label % 2 == 0), (label >= 0) & (label % 2 == 1)
    assert logp[good].mean() > ref[good].mean() + 1.0 and logp[bad].mean() < ref[bad].mean()
    assert totals.isfinite().all()


def test_preference_steps_separate_the_pairs(zs, cuda_device):
    import finetune_step
    totals, _, _, _, ctrl = finetune_step.run("preference", steps=24)
    assert ctrl["step"] == 24 and ctrl["skipped"] == 0
    assert totals[-1, 0] < 0.5 * totals[0, 0]               # from ln 2
    assert totals[0, 1] == 0.0 and totals[-1, 1] > 0.95     # every pair in order


def test_example_is_repeatable(zs, cuda_device):
    import finetune_step
    a, b = finetune_step.run("preference", steps=5)[0], finetune_step.run("preference", steps=5)[0]
    # (index_add_ of the embedding's gradient adds in no fixed order: bf16 sums)
    assert (a - b).abs().max() < 1e-2


def test_loss_suites_under_index_checks(zs, cuda_device):
    from zero_partitioned_mixed_partition_gb300 import build
    build.build(checked=True)
    env = dict(os.environ, ZS_CHECKED="1")
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "-k", "not past_32",
           *[os.path.join(ROOT, "tests", f) for f in ("test_gpu_losses.py", "test_gpu_tensors.py")]]
    r = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    tail = "\n".join((r.stdout + r.stderr).strip().splitlines()[-15:])
    assert r.returncode == 0, tail
    assert " passed" in tail and "failed" not in tail, tail
