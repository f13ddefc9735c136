"""The cache of cluster counts (csrc/cluster_counts.h) against a fake query: an
answer is kept for its device, kernel and shape, a failure is not kept."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include "cluster_counts.h"

int main() {
    zs::ClusterCounts counts;
    int asked = 0, bad = 0, answer = 0;
    auto query = [&] { ++asked; return answer; };
    int k[2];
    auto expect = [&](int device, const void* kernel, int ctas, int smem, int want, int want_asked) {
        const int got = counts.get(device, kernel, ctas, smem, query);
        if (got != want || asked != want_asked) {
            std::printf("device %d, ctas %d, smem %d: %d after %d queries, expected %d after %d\n", device, ctas, smem, got, asked, want, want_asked);
            ++bad;
        }
    };
    expect(0, &k[0], 2, 100, 0, 1);    // a failure is passed on
    answer = -1;
    expect(0, &k[0], 2, 100, -1, 2);   // and not kept
    answer = 148;
    expect(0, &k[0], 2, 100, 148, 3);
    answer = 20;
    expect(0, &k[0], 2, 100, 148, 3);  // a count is
    expect(1, &k[0], 2, 100, 20, 4);   // for its device,
    expect(0, &k[1], 2, 100, 20, 5);   // kernel,
    expect(0, &k[0], 4, 100, 20, 6);   // cluster size
    expect(0, &k[0], 2, 200, 20, 7);   // and shared memory
    answer = 7;
    expect(0, &k[0], 2, 100, 148, 7);
    expect(1, &k[0], 2, 100, 20, 7);
    std::puts(bad ? "failed" : "ok");
    return bad;
}
"""


def test_cluster_counts(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("needs g++")
    src, exe = tmp_path / "check.cpp", tmp_path / "check"
    src.write_text(PROGRAM)
    csrc = os.path.join(ROOT, "zero_partitioned_mixed_partition_gb300", "csrc")
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-I", csrc, str(src), "-o", str(exe), "-lpthread"], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
