"""The walk of the streaming products over their units, on the CPU: the arithmetic that the kernels share with the
host, compiled as plain C++."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_scaled_mxfp4_bf16_gb300", "csrc")
CUDA_INC = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")

HARNESS = r"""
#include <cmath>
#include <cstdio>
#include <random>
#include "stream.h"
using namespace mxfp4;
int main() {
    std::mt19937_64 rng(1);
    auto log_int = [&](double hi) { return (int64_t)std::exp2(std::generate_canonical<double, 53>(rng) * std::log2(hi)); };
    for (int k = 0; k < 4000000; ++k) {
        // any weight tiles that N < 2^31 makes, any token tiles that keep the units below 2^31
        const int64_t n_tiles = k % 4 ? log_int(1 << 24) : (1 << 24) - (int64_t)(rng() % 1000);
        const int64_t tiles = log_int((double)((int64_t(1) << 31) - 1) / n_tiles);
        int64_t r = rng() % (n_tiles * tiles);
        if (k % 3 == 0) r = r / tiles * tiles;                      // a weight tile's first and last unit
        if (k % 3 == 1) r = r / tiles * tiles + tiles - 1;
        const int nt = quotient_by_tiles((int)r, (int)tiles, tile_reciprocal((int)tiles), 0);
        if (nt != r / tiles) {
            printf("unit %ld of %ld x %ld tiles: weight tile %d\n", (long)r, (long)n_tiles, (long)tiles, nt);
            return 1;
        }
        // a group's rows to a token tile
        const int m_tile = (const int[]){32, 128, 192}[k % 3], n = k % 5 ? (int)log_int(1 << 30) : (1 << 30) - (int)(rng() % 5000);
        const int t = tiles_of(n, m_tile), per = 16 * (quotient_by_tiles(n - 1, 16 * t, tile_reciprocal(t), 4) + 1);
        if (per != tile_rows(n, m_tile)) {
            printf("%d rows in tiles of %d: %d a tile\n", n, m_tile, per);
            return 1;
        }
    }
    puts("ok");
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs the host C++ compiler")
def test_quotients_by_a_groups_tiles_are_exact(tmp_path):
    src = tmp_path / "walk.cpp"
    src.write_text(HARNESS)
    exe = tmp_path / "walk"
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", CSRC, "-I", CUDA_INC, "-o", str(exe), str(src)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert out.stdout.strip() == "ok", out.stdout
