"""Where the pieces of a sum over K start, at the largest sizes that are taken:
checked without a GPU, the header compiled for the host."""
import os
import re
import shutil
import subprocess

import pytest

from test_devices_cpu import CSRC, cuda_include

LARGEST = (2 ** 31 - 4096) // 4          # hidden sizes above it are refused

PROGRAM = r"""
#include "split.cuh"
#include <cstdio>

int main() {
    int total, part, parts;
    while (scanf("%d %d %d", &total, &part, &parts) == 3) {
        printf("%d\n", tcg::run_start(total, part, parts));
        tcg::Pieces of(total, parts);
        for (int round = 0; round < 2; ++round)
            for (int i = 0; i < parts; ++i) {
                of.next();
                if (of.begin != tcg::run_start(total, i, parts) || of.end != tcg::run_start(total, i + 1, parts)) return 1;
            }
    }
    return 0;
}
"""


def test_pieces_of_the_longest_sums(tmp_path):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "split.cpp", tmp_path / "split"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-w", "-I", CSRC, "-I", cuda_include(), "-o", str(exe), str(src)], check=True)
    asked = []
    for hidden in (1, 64, 1535, 1536, 4096, 11_900_000, 12_000_008, 16_800_008, LARGEST - 1, LARGEST):
        parts = max(1, (hidden + 512) // 1024)
        for stage in (64, 128):          # k a stage: one CTA, a pair
            total = -(-hidden // stage)
            n = min(parts, total)
            asked += [(total, p, n) for p in sorted({0, 1, n // 3, n // 2, n - 1, n})]
    asked += [(2 ** 31 - 1, p, 1024) for p in (0, 1, 1023, 1024)]
    out = subprocess.run([str(exe)], input="\n".join("%d %d %d" % a for a in asked), capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in out] == [t * p // n for t, p, n in asked]


def test_no_product_of_stages_and_parts_in_32_bits():
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        assert not re.search(r"(?<!>\()\b(?:p\.)?num_kb \* \(?(?:v\.)?(?:part|split)\b", text), name
