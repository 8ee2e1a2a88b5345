"""The ranges of a layer's split sums, on the CPU: a plain C++ program prints those that
the kernels' own header gives (csrc/layer_ranges.hpp)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include "layer_ranges.hpp"
#include <stdio.h>
#include <stdlib.h>
int main(int argc, char **argv)
{
    for (int a = 1; a + 1 < argc; a += 2) {
        const int n = atoi(argv[a]), splits = atoi(argv[a + 1]);
        for (int i = 0; i < splits; ++i) {
            int32_t first, length;
            dg::range_of(n, splits, i, first, length);
            printf("%d %d ", first, length);
        }
        printf("\n");
    }
}
"""
MOST = 2 ** 31 - 1025          # the longest sum that the calls take
LENGTHS = [0, 1, 63, 64, 65, 1000, 4096, 70001, 2 ** 26 + 1, MOST - 3071, MOST - 3070, MOST - 64, MOST - 1, MOST]
RANGES = [2, 3, 16, 1000, 1025, 1026, 1027, 2048, 4095, 4096]


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ is not installed")
def test_ranges_cover_the_sum(tmp_path):
    src, exe = tmp_path / "ranges.cpp", tmp_path / "ranges"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-ftrapv", "-I", os.path.join(ROOT, "dense_gemm_amd", "csrc"), str(src), "-o", str(exe)],
                   check=True)
    cases = [(n, s) for n in LENGTHS for s in RANGES]
    out = subprocess.run([str(exe)] + [str(x) for c in cases for x in c], check=True, capture_output=True, text=True).stdout.splitlines()
    assert len(out) == len(cases)
    for (n, s), line in zip(cases, out):
        v = [int(x) for x in line.split()]
        chunk = -(-(-(-n // s)) // 64) * 64                  # in Python's integers
        want = [(min(i * chunk, n), min(chunk, n - min(i * chunk, n))) for i in range(s)]
        assert list(zip(v[::2], v[1::2])) == want, (n, s)
        assert sum(v[1::2]) == n
