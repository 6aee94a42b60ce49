"""The grid of a product of few tokens with int8 weights: one CTA takes an SM, so a grid of more
than the SMs takes twice as long.  A host program over the library's own rule (wcols_runs.h)."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "verifiable_quantize_rows_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <initializer_list>
#include "wcols_runs.h"
int main() {
    for (long long sms = 1; sms <= 256; ++sms)
        for (long long blocks = 1; blocks <= 16; ++blocks)
            for (long long all : {1LL, 2LL, 7LL, 50LL, 51LL, 1024LL, 1LL << 33}) {
                const long long runs = bsg::wcols_runs(all, blocks, sms);
                if (runs < 1 || runs > all) return std::printf("runs %lld of %lld\n", runs, all), 1;
                if (blocks <= sms && runs * blocks > sms) return std::printf("%lld SMs: %lld x %lld\n", sms, runs, blocks), 1;
                // no SM without need idle: one run more would not fit
                if (blocks <= sms && runs < all && (runs + 1) * blocks <= sms) return std::printf("%lld SMs: only %lld x %lld\n", sms, runs, blocks), 1;
            }
    std::puts("ok");
}
"""


def test_no_more_ctas_than_sms(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    (tmp_path / "walk.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-I", CSRC, "-o", str(tmp_path / "walk"), str(tmp_path / "walk.cpp")], check=True, capture_output=True, text=True)
    r = subprocess.run([str(tmp_path / "walk")], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout


def test_the_launch_goes_by_the_rule():
    text = open(os.path.join(CSRC, "wcols.cu")).read()
    assert "cfg.gridDim = dim3((unsigned)wcols_runs(a.all, blocks, sms), (unsigned)blocks);" in text
