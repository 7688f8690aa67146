"""Blocks of 128 along a side up to the last that an int holds (csrc/f8_kernels.h), without a GPU: the
host's arithmetic, compiled as the library compiles it, with overflow made to show."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SIDES = [1, 16, 127, 128, 129, 2880, (1 << 24) + 16, 2147483504, 2147483520, 2147483521, 2147483536, 2147483632, 2147483647]


def test_blocks_of_a_side(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc) or shutil.which("g++") is None:
        pytest.skip("no compiler")
    src = tmp_path / "blocks.cpp"
    src.write_text('#include <cstdio>\n#include "f8_kernels.h"\nint main(int c, char** v) {\n'
                   '  for (int i = 1; i < c; ++i) { int n; std::sscanf(v[i], "%d", &n); std::printf("%d ", mxk::f8_blocks(n)); }\n}\n')
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=signed-integer-overflow", "-fsanitize-undefined-trap-on-error", "-I", include, "-I",
                    os.path.join(ROOT, "mxfp4_dequant_matmul_gb300", "csrc"), str(src), "-o", str(tmp_path / "blocks")], check=True)
    run = subprocess.run([str(tmp_path / "blocks")] + [str(n) for n in SIDES], capture_output=True, text=True)
    assert run.returncode == 0 and [int(b) for b in run.stdout.split()] == [-(-n // 128) for n in SIDES], run
