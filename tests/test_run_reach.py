"""How far a run of equal keys goes on (csrc/run_reach.h), against a walk, and how often the
list is looked at for it: once for a short run, and 2 log_32 of its length and a few at most."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include "run_reach.h"

int main() {
    int bad = 0;
    auto check = [&](int64_t run, int64_t list) {  // a run of `run` places in a list that ends after `list`
        int looks = 0;
        const int64_t want = run < list ? run : list;
        const int64_t got = zs::run_reach([&](int64_t at, int64_t stride) {
            ++looks;
            uint32_t bits = 0;
            for (int i = 0; i < 32; ++i) bits |= (uint32_t)(at + stride * (i + 1) <= want) << i;
            return bits;
        });
        int most = 1;
        for (int64_t n = want; n >= 32; n /= 32) most += 2;
        if (got != want || looks > most + 2 || (want < 32 && looks != 1)) {
            std::printf("%lld of %lld: %lld in %d looks\n", (long long)run, (long long)list, (long long)got, looks);
            ++bad;
        }
    };
    for (int64_t run = 0; run < 70000; ++run) check(run, 1ll << 40);
    for (int64_t run = 0; run < 3000; ++run) check(1ll << 40, run);
    for (int64_t run = 1; run < 1ll << 26; run = run * 5 / 4 + 1)
        for (int64_t d = -1; d <= 1; ++d) check(run + d, 1 << 25);
    std::puts(bad ? "failed" : "ok");
    return bad != 0;
}
"""


def test_run_reach(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("needs g++")
    src, exe = tmp_path / "check.cpp", tmp_path / "check"
    src.write_text(PROGRAM)
    csrc = os.path.join(ROOT, "zero_partitioned_mixed_partition_gb300", "csrc")
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-I", csrc, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
