"""Argument checks of the mixture-of-experts and weight-only operators, on the CPU: the C entry
points refuse bad arguments before they ask for a device, and the binding refuses tensors that would
make the kernels read or write past a buffer. And the tiling arithmetic the host and the kernels
share, compiled as plain C++."""
import os
import shutil
import subprocess

import pytest
import torch

import block_scaled_mxfp4_bf16_gb300 as mx
from block_scaled_mxfp4_bf16_gb300 import moe
from test_binding_checks import _Lib, dev

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_scaled_mxfp4_bf16_gb300", "csrc")
CUDA_INC = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")

OK, ARG, SHAPE, ALIGN = 0, 1, 2, 3
P = 1 << 20      # an aligned pointer that is never followed


@pytest.fixture(scope="module")
def c():
    return mx.load_library()


def test_gemv_refusals(c):
    def call(x=P, M=2, K=256, ldx=256, b=P, N=128, y=P, ldy=128, ws=P, n=1 << 30):
        return c.mxfp4_gemv(x, M, K, ldx, b, N, y, ldy, ws, n, None)
    assert call(M=-1) == call(N=-1) == call(K=-8) == ARG
    assert call(K=0) == call(K=12) == call(ldx=248) == call(ldy=127) == SHAPE
    assert call(N=1 << 31, ldy=1 << 31) == call(K=(1 << 30) + 8, ldx=1 << 40) == call(M=1 << 40) == SHAPE
    assert call(x=None) == call(b=None) == call(y=None) == ARG
    assert call(x=P + 8) == call(ldx=260) == call(b=P + 512) == call(y=P + 1) == ALIGN
    assert call(M=0) == call(N=0, ldy=0) == OK
    assert c.mxfp4_gemv_workspace_size(0, 128, 256) == c.mxfp4_gemv_workspace_size(1, 128, 12) == 0


def test_grouped_refusals(c):
    def call(a=P, t=8, K=256, lda=256, rows=None, off=P, E=4, b=P, N=128, out=P, R=8, ldc=128, flags=0, ws=P, n=1 << 30):
        return c.mxfp4_grouped_gemm(a, t, K, lda, rows, off, E, b, N, out, R, ldc, flags, ws, n, None)
    assert call(t=-1) == call(R=-1) == call(E=-1) == call(N=-1) == call(K=-8) == call(flags=2) == ARG
    assert call(K=0) == call(K=4) == call(lda=248) == call(ldc=100) == call(E=1025) == call(R=1 << 31, t=1 << 31) == SHAPE
    assert call(t=7) == SHAPE                       # without rows, one row of C per row of A
    assert call(flags=1) == SHAPE                   # gated rows are 2K long
    assert call(a=None) == call(off=None) == call(b=None) == call(out=None) == ARG
    assert call(a=P + 2) == call(lda=257) == call(b=P + 16) == call(out=P + 1) == call(rows=P + 2) == call(off=P + 2) == ALIGN
    assert call(R=0, t=0) == call(N=0, ldc=0) == call(E=0) == OK
    for bad in ((0, 4, 128, 256), (8, 0, 128, 256), (8, 1025, 128, 256), (8, 4, 0, 256), (8, 4, 128, 100)):
        assert c.mxfp4_grouped_gemm_workspace_size(*bad) == 0


def test_route_refusals(c):
    def call(x=P, dt=0, T=4, E=16, ld=16, k=2, flags=0, w=P, e=P, o=P, r=P, s=P, ws=P, n=1 << 20):
        return c.mxfp4_moe_route(x, dt, T, E, ld, k, flags, w, e, o, r, s, ws, n, None)
    assert call(T=-1) == call(E=0) == call(k=0) == call(dt=2) == call(flags=2) == ARG
    assert call(E=1025, ld=1025) == call(k=17) == call(E=64, ld=64, k=33) == call(ld=15) == call(T=1 << 30) == SHAPE
    for name in ("x", "w", "e", "o", "r", "s"):
        assert call(**{name: None}) == ARG
    assert call(x=P + 2) == call(w=P + 1) == call(r=P + 2) == ALIGN
    assert call(x=P + 1, dt=1) == ALIGN


def test_combine_refusals(c):
    def call(y=P, R=8, N=64, ldy=64, s=P, w=P, T=4, k=2, out=P, ldo=64):
        return c.mxfp4_moe_combine(y, R, N, ldy, s, w, T, k, out, ldo, None)
    assert call(R=-1) == call(N=-1) == call(T=-1) == call(k=-1) == ARG
    assert call(ldy=63) == call(ldo=63) == call(T=1 << 31) == SHAPE
    assert call(y=None) == call(s=None) == call(w=None) == call(out=None) == ARG
    assert call(y=P + 1) == call(out=P + 1) == call(s=P + 2) == call(w=P + 2) == ALIGN
    assert call(T=0) == call(N=0, ldy=0, ldo=0) == OK


class _MoeLib(_Lib):
    COMPUTE = _Lib.COMPUTE + ("mxfp4_gemv", "mxfp4_grouped_gemm", "mxfp4_moe_route", "mxfp4_moe_combine")
    SIZES = ("mxfp4_gemv_workspace_size", "mxfp4_grouped_gemm_workspace_size", "mxfp4_moe_route_workspace_size")

    def __getattr__(self, name):
        if name in self.SIZES:
            return lambda *a: 4096
        return super().__getattr__(name)


@pytest.fixture
def lib(monkeypatch):
    fake = _MoeLib(mx.load_library())
    monkeypatch.setattr(mx, "load_library", lambda: fake)
    monkeypatch.setattr(moe, "load_library", lambda: fake)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)   # a CPU tensor's get_device()
    monkeypatch.setattr(moe, "_NEED", {})
    return fake


def bf16(*shape):
    return dev(torch.zeros(*shape, dtype=torch.bfloat16))


def i32(*values):
    return dev(torch.tensor(values, dtype=torch.int32))


def ws():
    return dev(torch.zeros(4096, dtype=torch.uint8))


def packed(E, N, K):
    return dev(torch.zeros(E, mx.mxfp4_prepack_b_size(N, K), dtype=torch.uint8))


def test_binding_gemv(lib):
    good = dict(x=bf16(2, 256), packed_b=packed(1, 128, 256)[0], N=128, y=bf16(2, 128), workspace=ws(), stream=0)
    mx.mxfp4_gemv(**good)
    name, args = lib.calls[-1]
    assert name == "mxfp4_gemv" and args[1:4] == (2, 256, 256) and args[5] == 128 and args[7] == 128
    for change in (dict(x=bf16(2, 256).float()), dict(x=bf16(256, 2).T), dict(x=bf16(256)),
                   dict(packed_b=packed(1, 100, 256)[0][:1000]), dict(y=bf16(2, 127)), dict(y=bf16(128, 2).T),
                   dict(x=torch.zeros(2, 256, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            mx.mxfp4_gemv(**{**good, **change})
    assert len(lib.calls) == 1


def test_binding_grouped(lib):
    good = dict(a=bf16(5, 256), packed_b=packed(3, 128, 256), offsets=i32(0, 2, 4, 6), N=128,
                rows=i32(0, 1, 2, 3, 4, 0), c=bf16(6, 128), workspace=ws(), stream=0)
    mx.mxfp4_grouped_gemm(**good)
    args = lib.calls[-1][1]
    assert args[1:4] == (5, 256, 256) and args[6] == 3 and args[10] == 6 and args[12] == 0
    mx.mxfp4_grouped_gemm(**{**good, "a": bf16(6, 512), "rows": None, "gated": True})
    args = lib.calls[-1][1]
    assert args[1:4] == (6, 256, 512) and args[4] is None and args[12] == 1
    for change in (dict(offsets=i32(0, 2, 4)), dict(offsets=i32(0, 2, 4, 6).long()), dict(rows=i32(0, 1).view(1, 2)),
                   dict(rows=i32(0, 1, 2, 3, 4, 0).long()), dict(packed_b=packed(3, 128, 256).view(-1)),
                   dict(packed_b=packed(3, 128, 256)[:, ::2]), dict(packed_b=packed(3, 256, 256)),
                   dict(c=bf16(5, 128)), dict(rows=None), dict(gated=True, a=bf16(5, 255)), dict(a=bf16(5, 256).half())):
        with pytest.raises(ValueError):
            mx.mxfp4_grouped_gemm(**{**good, **change})
    assert len(lib.calls) == 2


def test_binding_route_and_combine(lib):
    for bad in (dict(logits=dev(torch.zeros(5, 16).half()), k=2), dict(logits=dev(torch.zeros(5, 16)), k=0),
                dict(logits=dev(torch.zeros(5, 16)), k=17), dict(logits=dev(torch.zeros(5, 64)), k=33),
                dict(logits=dev(torch.zeros(16, 5)).T, k=2), dict(logits=dev(torch.zeros(16)), k=2)):
        with pytest.raises(ValueError):
            mx.mxfp4_moe_route(**bad, stream=0)
    slots = i32(0, 1, 2, 3).view(2, 2)
    w = dev(torch.zeros(2, 2))
    mx.mxfp4_moe_combine(bf16(4, 64), slots, w, out=bf16(2, 64), stream=0)
    args = lib.calls[-1][1]
    assert args[1:4] == (4, 64, 64) and args[6:8] == (2, 2)
    for bad in (dict(y=bf16(4, 64).float(), slots=slots, weights=w), dict(y=bf16(4, 64), slots=slots.long(), weights=w),
                dict(y=bf16(4, 64), slots=slots, weights=dev(torch.zeros(2, 3))),
                dict(y=bf16(4, 64), slots=slots.view(4), weights=w),
                dict(y=bf16(4, 64), slots=slots, weights=w.to(torch.bfloat16)),
                dict(y=bf16(4, 64), slots=slots, weights=w, out=bf16(2, 63))):
        with pytest.raises(ValueError):
            mx.mxfp4_moe_combine(**bad, stream=0)
    assert len(lib.calls) == 1


HARNESS = r"""
#include <cstdio>
#include <random>
#include <set>
#include <vector>
#include "stream.h"
using namespace mxfp4;
int main() {
    std::mt19937 rng(1);
    for (int m_tile : {32, 64, 128, 192}) {
        // every group size: the tiles cover it exactly, each within the tile and not empty
        for (int n = 1; n <= 5000; ++n) {
            const int tiles = tiles_of(n, m_tile), per = tile_rows(n, m_tile);
            if (per % 16 || per > m_tile || (tiles - 1) * per >= n || tiles * per < n) { printf("rows %d %d\n", m_tile, n); return 1; }
        }
        // tile slots of all groups: distinct and below the bound
        for (int round = 0; round < 300; ++round) {
            const int groups = 1 + rng() % 200;
            std::vector<int> sizes(groups);
            int64_t rows = 0;
            for (int& s : sizes) { s = rng() % 3 == 0 ? 0 : rng() % (1 + rng() % 700); rows += s; }
            std::set<int> seen;
            int begin = 0;
            for (int g = 0; g < groups; ++g) {
                for (int i = 0; i < tiles_of(sizes[g], m_tile); ++i)
                    if (tile_slot(begin, g, i, m_tile) >= stream_tile_bound(rows, groups, m_tile) ||
                        !seen.insert(tile_slot(begin, g, i, m_tile)).second) { printf("slot %d\n", m_tile); return 1; }
                begin += sizes[g];
            }
        }
    }
    puts("ok");
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs the host C++ compiler")
def test_tiles_cover_every_group_and_their_slots_are_distinct(tmp_path):
    src = tmp_path / "tiles.cpp"
    src.write_text(HARNESS)
    exe = tmp_path / "tiles"
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, "-I", CUDA_INC, "-o", str(exe), str(src)], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True).stdout.strip() == "ok"


PLAN_HARNESS = r"""
#include <algorithm>
#include <cstdio>
#include <random>
#include "stream.h"
using namespace mxfp4;
static int clusters(int s) { return s == 1 ? 152 : 144 / s; }
#define CHECK(x) do { if (!(x)) { printf("%s: rows %ld groups %ld N %ld K %ld terms %d\n", #x, (long)rows, (long)groups, (long)N, (long)K, terms); return 1; } } while (0)
int main() {
    std::mt19937 rng(1);
    auto log_int = [&](double hi) { return (int64_t)std::exp2(std::generate_canonical<double, 32>(rng) * std::log2(hi)); };
    for (int i = 0; i < 200000; ++i) {
        const int terms = i % 2 ? kTerms : 1;
        const int64_t groups = terms > 1 ? 1 : log_int(1024), N = log_int(200000), K = 8 * log_int(4000);
        const int64_t rows = terms > 1 ? kTerms * (i % 4 == 1 ? log_int(40) : 1 + rng() % 16) : log_int(60000);
        StreamPlan p;
        CHECK(make_stream_plan(rows, groups, N, K, terms, 152, clusters, &p) == 0);
        // shared memory: everything the kernel lays out, within the limit, and (but for 2 KB) as large a
        // part of the SM's as the columns are of its tensor memory
        const uint32_t t_stage = p.pair ? p.a_block - p.m_tile * 64 : p.a_block;
        const size_t laid = 1024 + (size_t)p.stages * (kWBlock + t_stage) + (p.pair ? 64 : 0) + ((p.pair ? 3 : 2) * kStreamMaxStages + 4) * 8 + 32 + 64 +
                            8 * kEpiStage + 2 * (groups + 1) * 4 + (size_t)(p.cluster > 1 ? p.cluster : 0) * (p.m_tile / terms) * kTileN * 4;
        CHECK(p.smem_bytes >= laid && p.smem_bytes <= kSmemLimit);
        CHECK((p.smem_bytes + 1024 + 2048) * 512 >= (size_t)233472 * p.tmem_cols);
        CHECK(p.stages >= 1 && p.stages <= kStreamMaxStages);
        const int sf_cols = p.pair ? kPairSfSlots * (int)kPairSfCols : p.stages * 8 * (1 + p.nmc);
        CHECK(p.accs * p.m_tile + sf_cols <= (int)p.tmem_cols && p.tmem_cols <= 512);
        if (p.pair) CHECK(terms == 1 && p.ctas % 2 == 0 && p.nmc == 2 && p.stages >= kPairSfSlots && p.cluster == 1 && p.accs == 2);
        CHECK(p.a_block == (uint32_t)(p.m_tile * 128 + p.nmc * 1024) && p.m_tile % 16 == 0 && p.m_tile <= 192);
        if (terms == 1) CHECK(p.cluster == 1 && p.accs == 2);
        // CTAs: one per SM at most, or whole clusters that are all resident, at least two steps each
        if (p.cluster > 1) CHECK(p.ctas == tiles_of((int)rows, p.m_tile) * p.n_tiles * p.cluster &&
                                 p.ctas / p.cluster <= clusters(p.cluster) && p.k_atoms >= 2 * p.cluster);
        else CHECK(p.ctas >= 1 && p.ctas <= 152);
        if (p.accs == 1 && p.cluster == 1) {   // every CTA really has one share: whole units, one each
            const int64_t units = (int64_t)tiles_of((int)rows, p.m_tile) * p.n_tiles, steps = units * p.k_atoms;
            const int64_t share = std::max<int64_t>((steps + p.ctas - 1) / p.ctas, (p.k_atoms + 5) / 6);
            CHECK(units <= p.ctas && (units == p.ctas || share + kSplitSteps > p.k_atoms));
        }
        // the fused kernels keep a row index per lane
        if (p.fused && terms == 1) CHECK(p.m_tile <= 32);
        CHECK(p.ws_total >= p.off_partial && p.off_partial >= p.off_counters + (size_t)p.ctas * 8);
    }
    puts("ok");
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs the host C++ compiler")
def test_plans_fit_the_sm_and_agree_with_the_kernel(tmp_path):
    from block_scaled_mxfp4_bf16_gb300 import build
    lib = build.build()
    src = tmp_path / "plan.cpp"
    src.write_text("#include <cmath>\n" + PLAN_HARNESS)
    exe = tmp_path / "plan"
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, "-I", CUDA_INC, "-o", str(exe), str(src), lib,
                    f"-Wl,-rpath,{os.path.dirname(lib)}"], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.stdout.strip() == "ok", out.stdout + out.stderr


def _expand(x, terms=8):
    """The weight-only product's expansion of one block, in Python: uniform steps on exact fractions."""
    from fractions import Fraction
    grid = sorted({s * m for m in (0, 0.5, 1, 1.5, 2, 3, 4, 6) for s in (1, -1)})
    import math
    amax = max(abs(v) for v in x)
    mant, expo = math.frexp(amax)                  # amax = mant * 2^expo, mant in [0.5, 1)
    s = expo - 1 + (1 if mant * 2 > 1.5 else 0) - 2
    rest = [Fraction(v) for v in x]
    for t in range(terms):
        step = Fraction(2) ** s
        rest = [r - step * Fraction(min(grid, key=lambda q: (abs(r / step - Fraction(q)), abs(q)))) for r in rest]
        s -= 2 if t == 0 else 3
    return max(abs(r) for r in rest) / Fraction(amax)


def test_the_expansion_holds_a_block_to_its_bound():
    g = torch.Generator().manual_seed(0)
    for i in range(40):
        x = (torch.randn(32, generator=g) * (10.0 ** (i % 7 - 3))).to(torch.bfloat16).float()
        if i % 5 == 0:
            x[3] *= 500
            x = x.to(torch.bfloat16).float()
        assert _expand(x.tolist()) <= 2.0 ** -22
    # every mantissa of the maximum against elements at the midpoints it leaves
    for m in range(128, 256):
        assert _expand([float(m), m * 0.625, m * 0.0390625, 1.0, 5.0 / 16, m / 2.0]) <= 2.0 ** -22
