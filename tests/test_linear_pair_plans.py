"""The shapes of test_gpu_linear_pairs run on pairs of CTAs, in the token tiles and with the cuts along K noted there:
the choice between a dense product's plans, compiled as plain C++, on the plans that the GEMM has for a GB300."""
import shutil
import subprocess

import pytest

import block_scaled_mxfp4_bf16_gb300 as mx
from test_gpu_linear_pairs import GATED_PAIRS, PAIRS
from test_moe_checks import CSRC, CUDA_INC
from test_planner import CLUSTER_CAPS, SM_COUNT

# Lines of M, N, K, the output's columns and the GEMM's CTAs, splits and token tile -> whether CTAs work in pairs, the
# token tile, whether the walk through the units cuts some of them along K (as begin_walk does).
HARNESS = r"""
#include <cstdio>
#include "stream.h"
using namespace mxfp4;
int main() {
    long long M, N, K, columns, ctas, splits, m_tile, sms;
    while (scanf("%lld %lld %lld %lld %lld %lld %lld %lld", &M, &N, &K, &columns, &ctas, &splits, &m_tile, &sms) == 8) {
        const DenseChoice c = choose_dense(M, N, K, (int)columns, ctas, (int)splits, (int)m_tile, (int)sms);
        int cut = 0;
        if (c.streams) {
            const long long k = (K + 255) / 256, n_tiles = (N + 127) / 128, walkers = c.pair ? sms / 2 : sms;
            const long long units = tiles_of((int)M, c.m_tile) * (c.pair ? (n_tiles + 1) / 2 : n_tiles);
            const long long rest = units % walkers, even = (rest * k + walkers - 1) / walkers;
            long long share = split_share(even, (int)k);
            const long long apart = share + kSplitSteps < k ? share + kSplitSteps : k;
            if (units >= walkers && rest > 0 && even + kMergeSteps < apart) share = ((rest + walkers) * k + walkers - 1) / walkers;
            cut = rest > 0 && share % k != 0;
        }
        printf("%d %d %d\n", c.streams && c.pair ? 1 : 0, c.m_tile, cut);
    }
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs the host C++ compiler")
def test_the_pair_shapes_run_in_pairs(tmp_path):
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text(HARNESS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, "-I", CUDA_INC, "-o", str(exe), str(src)], check=True)
    cases = [(s, s[1], s[1], want) for s, want in PAIRS.items()]
    cases += [(s, 2 * ((s[1] + 7) // 8 * 8), s[1], want) for s, want in GATED_PAIRS.items()]
    lines = []
    for (M, _, K), N, columns, _ in cases:
        plan = mx.mxfp4_gemm_plan_model(M, N, K, SM_COUNT, CLUSTER_CAPS)
        assert plan["path"] == 2
        lines.append(f"{M} {N} {K} {columns} {plan['ctas']} {plan['splits']} {plan['m_tile']} {SM_COUNT}")
    out = subprocess.run([str(exe)], input="\n".join(lines), text=True, capture_output=True, timeout=60, check=True).stdout.split("\n")
    for (shape, _, _, (tile, cut)), line in zip(cases, out):
        assert line == f"1 {tile} {int(cut)}", (shape, line)
    # tensor copies and element stores both, each on whole and on cut units
    assert {(N % 8 == 0, cut) for (_, N, _), (_, cut) in PAIRS.items()} == {(True, True), (True, False), (False, True), (False, False)}
