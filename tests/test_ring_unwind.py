"""A block that gives up on a ring of copies stays until they have landed: the places that it waits
at, compiled for the host and played through, and where the kernels do it."""
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

// An mbarrier of one arrival: `done` phases are complete; a wait for a parity passes while the phase
// under way has the other one.
struct Barrier { int done; bool passes(uint32_t parity) const { return (uint32_t)(done & 1) != parity; } };

static bool landed(const Barrier* b, int stages, ito::RingPlace at, int copies)
{
    for (int i = 0; i < copies; ++i, at.next(stages))
        if (!b[at.stage].passes(at.phase)) return false;
    return true;
}

int main()
{
    int checks = 0;
    for (int stages = 1; stages <= 9; ++stages)
        for (int issued = 0; issued <= 4 * stages + 1; ++issued) {
            ito::RingPlace next{0, 0}, first{0, 0};
            for (int i = 0; i < issued; ++i) next.next(stages);
            const int there = issued < stages ? issued : stages;
            for (int i = 0; i < issued - there; ++i) first.next(stages);
            // the copies before the last lap have landed; of its own any subset may have
            for (int mask = 0; mask < 1 << there; ++mask) {
                Barrier b[9] = {};
                for (int i = 0; i < issued; ++i)
                    if (i < issued - there || (mask >> (i - (issued - there)) & 1)) ++b[i % stages].done;
                const bool all = mask == (1 << there) - 1;
                // a producer, from its next place; a consumer, from the first copy it has not seen
                if (landed(b, stages, next.lap_before(), stages) != all || landed(b, stages, first, there) != all) {
                    printf("stages %d issued %d mask %d\n", stages, issued, mask);
                    return 1;
                }
                ++checks;
            }
        }
    printf("%d\n", checks);
    return 0;
}
"""


@pytest.mark.skipif(not os.path.exists(NVCC), reason="nvcc not found")
def test_the_places_are_those_of_the_copies_under_way(tmp_path):
    src, exe = tmp_path / "play.cu", tmp_path / "play"
    src.write_text(PLAY)
    subprocess.run([NVCC, "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "--expt-relaxed-constexpr",
                    "-I" + CSRC, "-I" + os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True,
                   capture_output=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout
    assert int(out.stdout) > 10000


def kernels(name):
    """Bodies of a file's kernels, by name."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    parts = re.split(r"__global__ void[^;{]*?\s(k_\w+)\(", text)
    bodies = {}
    for kernel, rest in zip(parts[1::2], parts[2::2]):
        at = rest.index("{")
        depth, end = 0, at
        for end in range(at, len(rest)):
            depth += (rest[end] == "{") - (rest[end] == "}")
            if depth == 0:
                break
        bodies[kernel] = rest[at:end + 1]
    return bodies


@pytest.mark.parametrize("name", ["ito_adamw.cu", "ito_layer_norm.cu", "ito_logprobs.cu", "ito_fp_gemm.cu"])
def test_kernels_that_copy_wait_for_their_copies(name):
    found = 0
    for kernel, body in kernels(name).items():
        if "bulk_load(" in body or "tma_load_2d" in body:
            assert "ring_landed(" in body or "ln_unwind(" in body, kernel
            if "tc_commit" in body:      # the products that read the stages as well
                assert "ring_landed(full_bar" in body and "ring_landed(empty_bar" in body, kernel
            found += 1
    assert found
