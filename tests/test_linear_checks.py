"""Argument checks of the products with an epilogue, on the CPU: the C entry points refuse bad arguments before they
ask for a device, and the binding refuses tensors that would make the kernels read or write past a buffer. And the
arithmetic that the host and the kernels share, compiled as plain C++."""
import os
import shutil
import subprocess

import pytest
import torch

import block_scaled_mxfp4_bf16_gb300 as mx
from block_scaled_mxfp4_bf16_gb300 import linear, moe
from test_binding_checks import dev
from test_moe_checks import ALIGN, ARG, CSRC, CUDA_INC, OK, P, SHAPE, _MoeLib, bf16, i32, packed, ws


@pytest.fixture(scope="module")
def c():
    return mx.load_library()


def test_linear_refusals(c):
    def call(x=P, M=2, K=256, ldx=256, b=P, N=128, bias=P, bt=0, act=0, res=P, ldr=128, out=P, ldo=128, ws=P, n=1 << 30):
        return c.mxfp4_linear(x, M, K, ldx, b, N, bias, bt, act, res, ldr, out, ldo, ws, n, None)
    assert call(M=-1) == call(N=-1) == call(K=-8) == call(act=-1) == call(act=5) == call(bt=2) == ARG
    assert call(K=0) == call(K=12) == call(ldx=248) == call(ldo=127) == call(ldr=127) == SHAPE
    assert call(N=1 << 31, ldo=1 << 31, ldr=1 << 31) == call(K=(1 << 30) + 8, ldx=1 << 40) == call(M=1 << 31) == SHAPE
    assert call(x=None) == call(b=None) == call(out=None) == ARG
    assert call(x=P + 8) == call(ldx=260) == call(b=P + 512) == call(out=P + 1) == call(res=P + 1) == ALIGN
    assert call(bias=P + 2) == call(bias=P + 1, bt=1) == ALIGN
    assert call(M=0) == call(N=0, ldo=0, ldr=0) == OK
    for bad in ((0, 128, 256), (2, 0, 256), (2, 128, 12), (1 << 31, 128, 256)):
        assert c.mxfp4_linear_workspace_size(*bad) == 0


def test_gated_refusals(c):
    def call(x=P, M=2, K=256, ldx=256, b=P, I=64, bias=P, bt=0, act=2, out=P, ldo=64, ws=P, n=1 << 30):
        return c.mxfp4_gated_linear(x, M, K, ldx, b, I, bias, bt, act, out, ldo, ws, n, None)
    assert call(M=-1) == call(I=-1) == call(K=-8) == call(act=5) == call(bt=-1) == ARG
    assert call(K=0) == call(K=12) == call(ldx=248) == call(ldo=63) == call(I=1 << 30, ldo=1 << 30) == SHAPE
    assert call(x=None) == call(b=None) == call(out=None) == ARG
    assert call(x=P + 8) == call(ldx=260) == call(b=P + 512) == call(out=P + 1) == call(bias=P + 2) == ALIGN
    assert call(M=0) == call(I=0, ldo=0) == OK
    for bad in ((0, 64, 256), (2, 0, 256), (2, 64, 12)):
        assert c.mxfp4_gated_linear_workspace_size(*bad) == 0


def test_grouped_gated_refusals(c):
    def call(a=P, t=8, K=256, lda=256, rows=None, off=P, E=4, b=P, I=64, bias=P, bt=0, act=2, out=P, R=8, ldo=64, ws=P,
             n=1 << 30):
        return c.mxfp4_grouped_gated_linear(a, t, K, lda, rows, off, E, b, I, bias, bt, act, out, R, ldo, ws, n, None)
    assert call(t=-1) == call(R=-1) == call(E=-1) == call(I=-1) == call(K=-8) == call(act=9) == call(bt=2) == ARG
    assert call(K=0) == call(K=4) == call(lda=248) == call(ldo=60) == call(E=1025) == call(R=1 << 31, t=1 << 31) == SHAPE
    assert call(t=7) == SHAPE                       # without rows, one row of the output per row of a
    assert call(a=None) == call(off=None) == call(b=None) == call(out=None) == ARG
    assert call(a=P + 2) == call(lda=257) == call(b=P + 16) == call(out=P + 1) == call(rows=P + 2) == call(off=P + 2) == ALIGN
    assert call(bias=P + 2) == call(bias=P + 1, bt=1) == ALIGN
    assert call(R=0, t=0) == call(I=0, ldo=0) == call(E=0) == OK
    for bad in ((0, 4, 64, 256), (8, 0, 64, 256), (8, 1025, 64, 256), (8, 4, 0, 256), (8, 4, 64, 100)):
        assert c.mxfp4_grouped_gated_linear_workspace_size(*bad) == 0


def test_prepack_gated_sizes_and_refusals(c):
    # 16 packed rows for every eight features begun, in tiles of 128 rows
    assert mx.mxfp4_prepack_gated_size(64, 256) == 17408 == mx.mxfp4_prepack_gated_size(1, 8)
    assert mx.mxfp4_prepack_gated_size(65, 256) == 2 * 17408
    assert mx.mxfp4_prepack_gated_size(2884, 2040) == 46 * 8 * 17408
    assert mx.mxfp4_prepack_gated_size(0, 256) == mx.mxfp4_prepack_gated_size(64, 12) == 0
    assert mx.mxfp4_prepack_gated_size(1 << 30, 256) == 0 < mx.mxfp4_prepack_gated_size((1 << 30) - 8, 256)

    def call(q=P, s=P, I=64, K=256, out=P):
        return c.mxfp4_prepack_gated(q, s, I, K, out, None)
    assert call(I=0) == call(K=0) == call(q=None) == call(s=None) == call(out=None) == ARG
    assert call(K=12) == call(I=1 << 30) == SHAPE
    assert call(q=P + 8) == call(out=P + 512) == ALIGN


class _LinearLib(_MoeLib):
    COMPUTE = _MoeLib.COMPUTE + ("mxfp4_linear", "mxfp4_gated_linear", "mxfp4_grouped_gated_linear", "mxfp4_prepack_gated")
    SIZES = _MoeLib.SIZES + ("mxfp4_linear_workspace_size", "mxfp4_gated_linear_workspace_size",
                             "mxfp4_grouped_gated_linear_workspace_size")


@pytest.fixture
def lib(monkeypatch):
    fake = _LinearLib(mx.load_library())
    for module in (mx, moe, linear):
        monkeypatch.setattr(module, "load_library", lambda: fake)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)   # a CPU tensor's get_device()
    monkeypatch.setattr(moe, "_NEED", {})
    monkeypatch.setattr(linear, "_SIZES", {})
    return fake


def gated_packed(E, I, K):
    return dev(torch.zeros(E, mx.mxfp4_prepack_gated_size(I, K), dtype=torch.uint8))


def f32(*shape):
    return dev(torch.zeros(*shape))


def test_binding_linear(lib):
    good = dict(x=bf16(2, 256), packed_b=packed(1, 128, 256)[0], N=128, bias=f32(128), activation="gelu",
                residual=bf16(2, 128), out=bf16(2, 128), workspace=ws(), stream=0)
    mx.mxfp4_linear(**good)
    name, args = lib.calls[-1]
    assert name == "mxfp4_linear" and args[1:4] == (2, 256, 256) and args[5] == 128 and args[7:9] == (0, 3)
    assert args[10] == 128 and args[12] == 128
    mx.mxfp4_linear(**{**good, "bias": bf16(128), "activation": None, "residual": None})
    args = lib.calls[-1][1]
    assert args[7:9] == (1, 0) and args[9] is None
    for change in (dict(x=bf16(2, 256).float()), dict(x=bf16(256, 2).T), dict(x=bf16(256)),
                   dict(packed_b=packed(1, 100, 256)[0][:1000]), dict(out=bf16(2, 127)), dict(out=bf16(128, 2).T),
                   dict(out=f32(2, 128)), dict(bias=f32(127)), dict(bias=f32(128).half()), dict(bias=f32(256)[::2]),
                   dict(bias=f32(1, 128)), dict(activation="tanh"), dict(activation=2), dict(residual=bf16(2, 127)),
                   dict(residual=bf16(128, 2).T), dict(residual=f32(2, 128)), dict(residual=bf16(1, 128)),
                   dict(x=torch.zeros(2, 256, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            mx.mxfp4_linear(**{**good, **change})
    assert len(lib.calls) == 2


def test_binding_gated(lib):
    good = dict(x=bf16(2, 256), packed_gu=gated_packed(1, 100, 256)[0], I=100, bias=f32(200), out=bf16(2, 100),
                workspace=ws(), stream=0)
    mx.mxfp4_gated_linear(**good)
    name, args = lib.calls[-1]
    assert name == "mxfp4_gated_linear" and args[1:4] == (2, 256, 256) and args[5] == 100 and args[7:9] == (0, 2)
    for change in (dict(x=bf16(2, 256).float()), dict(packed_gu=gated_packed(1, 100, 256)[0][:20000]), dict(I=200),
                   dict(bias=f32(100)), dict(bias=f32(2, 100)), dict(out=bf16(2, 200)), dict(activation="swish")):
        with pytest.raises(ValueError):
            mx.mxfp4_gated_linear(**{**good, **change})
    assert len(lib.calls) == 1


def test_binding_grouped_gated(lib):
    good = dict(a=bf16(5, 256), packed_gu=gated_packed(3, 64, 256), offsets=i32(0, 2, 4, 6), I=64,
                rows=i32(0, 1, 2, 3, 4, 0), bias=bf16(3, 128), out=bf16(6, 64), workspace=ws(), stream=0)
    mx.mxfp4_grouped_gated_linear(**good)
    args = lib.calls[-1][1]
    assert args[1:4] == (5, 256, 256) and args[6] == 3 and args[8] == 64 and args[10:12] == (1, 2) and args[13] == 6
    for change in (dict(offsets=i32(0, 2, 4)), dict(offsets=i32(0, 2, 4, 6).long()), dict(rows=i32(0, 1).view(1, 2)),
                   dict(rows=i32(0, 1, 2, 3, 4, 0).long()), dict(packed_gu=gated_packed(3, 64, 256).view(-1)),
                   dict(packed_gu=gated_packed(3, 64, 256)[:, ::2]), dict(packed_gu=gated_packed(3, 128, 256)),
                   dict(out=bf16(5, 64)), dict(rows=None), dict(bias=bf16(128)), dict(bias=bf16(2, 128)),
                   dict(bias=bf16(3, 64)), dict(a=bf16(5, 256).half())):
        with pytest.raises(ValueError):
            mx.mxfp4_grouped_gated_linear(**{**good, **change})
    assert len(lib.calls) == 1


def test_binding_prepack_gated(lib):
    def u8(*shape):
        return dev(torch.zeros(*shape, dtype=torch.uint8))
    mx.mxfp4_prepack_gated(u8(200, 128), u8(200, 8), packed=gated_packed(1, 100, 256)[0], stream=0)
    name, args = lib.calls[-1]
    assert name == "mxfp4_prepack_gated" and args[2:4] == (100, 256)
    small = gated_packed(1, 100, 256)[0][:17408]
    for q, s, kw in ((u8(201, 128), u8(201, 8), {}), (u8(200, 128), u8(200, 7), {}), (u8(200, 128), u8(199, 8), {}),
                     (u8(128, 200).T, u8(200, 8), {}), (u8(200, 128).float(), u8(200, 8), {}),
                     (u8(200, 128), u8(200, 8), dict(packed=small)), (u8(1, 200, 128), u8(1, 200, 8), {})):
        with pytest.raises(ValueError):
            mx.mxfp4_prepack_gated(q, s, stream=0, **kw)
    with pytest.raises(ValueError):
        mx.mxfp4_prepack_gated_experts(u8(200, 128), u8(200, 8), stream=0)
    assert len(lib.calls) == 1


HARNESS = r"""
#include <cmath>
#include <cstdio>
#include <random>
#include <set>
#include "stream.h"
using namespace mxfp4;
int main() {
    // an owner's rows in the split-K sum of gated weights: whole sixteens, all 128 rows of the tile owned once
    for (int s = 1; s <= 16; ++s) {
        const int r = res_rows_per_owner(s, 16);
        if (r % 16 || r * s < kTileN || res_rows_per_owner(s, 1) != (kTileN + s - 1) / s) return 1;
    }
    // packed rows: every feature's two rows eight apart, all different, none past the end
    for (int I = 1; I < 300; ++I) {
        std::set<int64_t> seen;
        for (int r = 0; r < gated_rows(I); ++r) {
            const int f = (r >> 4) * 8 + (r & 7);
            if (f < I) seen.insert(f + ((r & 8) ? I : 0));
            else if (f >= (I + 7) / 8 * 8) return 2;
        }
        if ((int)seen.size() != 2 * I || gated_rows(I) % 16) return 3;
    }
    // stages of the pair kernel: the scale warps of set n % 2 wait for fill n / stages of stage n % stages by its parity
    // alone, having waited for step n - 2 - kPairSfSlots to be over at step n - 2; fills land in any order. Whatever fill
    // of the stage is the last to have landed then, it must not be taken for this one.
    for (int fit = 2; fit <= kStreamMaxStages; ++fit) {
        const int stages = pair_stages(fit);
        if (stages > fit || stages < fit - 1 || stages < 2) return 5;
        for (int n = 0; n < 200; ++n) {
            const int fill = n / stages, stage = n % stages, over = n - 2 - kPairSfSlots;
            // the set itself has seen every fill of the stage that was its own; others' are sure only if they are over
            int landed = 0;
            for (int f = 0; f < fill; ++f) {
                const int step = f * stages + stage;
                if (step <= over || step % 2 == n % 2) landed = f + 1;
            }
            if (landed < fill) return 6;          // with one fill less landed, the parity is that of a fill that is in
        }
    }
    if (pair_stages(5) != 4 || pair_stages(7) != 7 || pair_stages(6) != 6) return 7;
    // a dense product's token tiles: whole sixteens up to 192 that tile M the same way again, and cover it
    std::mt19937 rng(1);
    for (int i = 0; i < 200000; ++i) {
        auto log_int = [&](double hi) { return (int64_t)std::exp2(std::generate_canonical<double, 53>(rng) * std::log2(hi)); };
        const int64_t M = i < 5000 ? i + 1 : log_int(1 << 30), N = log_int(1 << 20), K = 8 * log_int(1 << 14);
        const int splits = 1 + (int)(rng() % 5), m_tile = 16 * (1 + (int)(rng() % 16));
        const DenseChoice c = choose_dense(M, N, K, (int)N, i % 3 ? 153 : 100, splits, m_tile, 152);
        if (!c.streams) {
            if (i % 3) return 4;      // the GEMM only where its CTAs make one wave
            continue;
        }
        if (c.m_tile < 16 || c.m_tile > 192 || c.m_tile % 16 || tile_rows((int)M, c.m_tile) != c.m_tile) return 8;
        const int64_t tiles = tiles_of((int)M, c.m_tile);
        if ((tiles - 1) * c.m_tile >= M || tiles * c.m_tile < M || (c.pair && (N <= 128 || K <= 7 * 256))) return 9;
    }
    puts("ok");
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs the host C++ compiler")
def test_shared_arithmetic(tmp_path):
    src = tmp_path / "linear.cpp"
    src.write_text(HARNESS)
    exe = tmp_path / "linear"
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", CSRC, "-I", CUDA_INC, "-o", str(exe), str(src)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.returncode
