"""The arrival counters of the streaming products' split units, on the CPU: the arithmetic that the kernels
share with the host, compiled as plain C++ and run for walkers that arrive in every order, some of which
gave up. A graph replays a launch with the same tag, so every run here has the same one."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_scaled_mxfp4_bf16_gb300", "csrc")
CUDA_INC = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")

HARNESS = r"""
#include <algorithm>
#include <cstdio>
#include <random>
#include "stream.h"
using namespace mxfp4;
int main() {
    std::mt19937_64 rng(1);
    const uint64_t tag = rng() >> 8;
    for (int i = 0; i < 200000; ++i) {
        const int walkers = 2 + (int)(rng() % 6);
        // what other uses of the workspace left there, with any low bits but not under this call's tag
        unsigned long long word = i % 3 ? rng() : 0ull;
        if ((word >> 8) == tag) word = 0ull;
        for (int replay = 0; replay < 4; ++replay) {
            const bool clean = replay % 2;
            int added = 0, lasts = 0, order[8] = {0, 1, 2, 3, 4, 5, 6, 7};
            std::shuffle(order, order + walkers, rng);
            bool any = false;
            for (int k = 0; k < walkers; ++k) {
                const bool gave_up = !clean && (rng() % 3 == 0 || order[k] == 0);
                any = any || gave_up;
                const bool ready = word == (tag << 8 | (unsigned)(walkers - 1));   // the others are there: no arrival needed
                if (ready && !gave_up) {
                    if (k != walkers - 1) { puts("early"); return 1; }
                    ++lasts;
                    ++added;
                    word = 0ull;
                    continue;
                }
                const unsigned long long mine = arrival_word(word, tag);
                word = arrival_add(mine, gave_up);
                if (arrival_last(mine, walkers - 1)) {
                    if (k != walkers - 1) { puts("last before its time"); return 1; }
                    ++lasts;
                    if (!gave_up && arrival_clean(mine)) ++added;
                    word = 0ull;
                }
            }
            if (lasts != 1 || added != (any ? 0 : 1) || word != 0ull) {
                printf("walkers %d replay %d: last %d added %d word %llx\n", walkers, replay, lasts, added, word);
                return 1;
            }
        }
    }
    puts("ok");
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs the host C++ compiler")
def test_a_unit_is_added_up_once_and_its_counter_left_cleared(tmp_path):
    src = tmp_path / "arrivals.cpp"
    src.write_text(HARNESS)
    exe = tmp_path / "arrivals"
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, "-I", CUDA_INC, "-o", str(exe), str(src)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert out.stdout.strip() == "ok", out.stdout
