"""What the library does once on each device, compiled for the host: a second device is not taken for the
first one, and what failed is done again."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "integer_only_nn_gb300", "csrc")
NVCC = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"

PLAY = r"""
#include <cstdio>
#include "ito_float.cuh"

int main()
{
    int calls = 0;
    ito::OnEachDevice once;
    auto ok = [&] { ++calls; return cudaSuccess; };
    auto bad = [&] { ++calls; return cudaErrorInvalidValue; };
    for (int turn = 0; turn < 3; ++turn)
        for (int device : {0, 1, 63})
            if (once.run(device, ok) != cudaSuccess) return 1;
    if (calls != 3) return 2;
    if (once.run(5, bad) != cudaErrorInvalidValue || calls != 4) return 3;
    if (once.run(5, ok) != cudaSuccess || calls != 5) return 4;
    if (once.run(5, bad) != cudaSuccess || calls != 5) return 5;
    // devices beyond the bits: every time
    if (once.run(64, ok) != cudaSuccess || once.run(64, ok) != cudaSuccess || calls != 7) return 6;
    return 0;
}
"""


@pytest.mark.skipif(not os.path.exists(NVCC), reason="nvcc not found")
def test_once_on_each_device(tmp_path):
    src, exe = tmp_path / "play.cu", tmp_path / "play"
    src.write_text(PLAY)
    subprocess.run([NVCC, "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "--expt-relaxed-constexpr",
                    "-I" + CSRC, "-I" + os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True,
                   capture_output=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_the_float_products_remember_nothing_for_all_devices():
    text = open(os.path.join(CSRC, "ito_fp_gemm.cu")).read()
    assert not re.search(r"static bool \w+ *[=;]", text) and text.count("static OnEachDevice") == 2
