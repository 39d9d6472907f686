"""How the streaming products cut what is left after their full waves, on the CPU: the plan (one accumulator for CTAs
that have one share) and the kernels take it from one function, held here against the rule it stands for."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_scaled_mxfp4_bf16_gb300", "csrc")
CUDA_INC = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")

HARNESS = r"""
#include <cstdio>
#include <random>
#include "stream.h"
using namespace mxfp4;
int main() {
    std::mt19937_64 rng(1);
    for (int i = 0; i < 300000; ++i) {
        const int k_atoms = 1 + (int)(rng() % (i % 2 ? 40 : 2000)), walkers = 1 + (int)(rng() % 160);
        const int64_t units = 1 + (int64_t)(rng() % walkers), steps = units * k_atoms;
        const int64_t share = split_share((steps + walkers - 1) / walkers, k_atoms);
        // all of the steps are somebody's, and a share is a unit at most
        if (share * walkers < steps || share < 1 || share > k_atoms) { printf("share %ld\n", (long)share); return 1; }
        // whole units, one each at most, or units cut where that saves eight steps
        if (share != k_atoms && share + kSplitSteps > k_atoms) { puts("a split that saves too little"); return 1; }
        for (int64_t u = 0; u < units; ++u) {
            const int64_t first = u * k_atoms / share, last = (u * k_atoms + k_atoms - 1) / share;
            if (last - first > 6) { puts("more than seven walkers to a unit"); return 1; }
            if (share == k_atoms && last != first) { puts("a whole unit of two walkers"); return 1; }
        }
    }
    puts("ok");
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs the host C++ compiler")
def test_shares_of_split_units(tmp_path):
    src = tmp_path / "share.cpp"
    src.write_text(HARNESS)
    exe = tmp_path / "share"
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, "-I", CUDA_INC, "-o", str(exe), str(src)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert out.stdout.strip() == "ok", out.stdout
