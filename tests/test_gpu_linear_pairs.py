"""The products with an epilogue on pairs of CTAs against 64-bit products: every activation, strides and starts off 16
bytes, in place on the residual, units that are cut along K. test_linear_pair_plans keeps these shapes on pairs."""
import pytest
import torch

from block_scaled_mxfp4_bf16_gb300 import workloads
from linear_testlib import ACTS, gated
from moe_testlib import assert_within, canary_out, outside_untouched, quantized, strided
from test_gpu_gated_linear import gated_weights, random_bias
from test_gpu_linear import check, operands

pytestmark = pytest.mark.gpu

# M, weight rows, K -> (token tile, units cut along K). Columns that are whole 16-byte pieces (tensor copies) and not.
PAIRS = {
    (538, 1072, 4536): (64, False), (2301, 2712, 2936): (192, False), (2576, 2760, 6696): (192, True),
    (1453, 5251, 3592): (160, False), (2578, 2692, 6064): (192, True),
}
# M, features, K of gated products (twice as many weight rows)
GATED_PAIRS = {(538, 536, 4536): (64, False), (2576, 1380, 6696): (192, True), (1453, 2625, 3592): (160, False)}


@pytest.mark.parametrize("activation", ACTS)
@pytest.mark.parametrize("M,N,K", PAIRS)
def test_activations(M, N, K, activation):
    import block_scaled_mxfp4_bf16_gb300 as mx
    packed, w, x, b, r = operands(M, N, K, torch.float32, True, seed=3)
    b = 10 * b                                          # far into both tails
    check(mx.mxfp4_linear(x, packed, N, bias=b, activation=activation), x, w, bias=b, activation=activation)
    out, store = canary_out(M, N, 0)
    mx.mxfp4_linear(x, packed, N, bias=b, activation=activation, residual=r, out=out)
    assert outside_untouched(out, store)
    check(out, x, w, bias=b, activation=activation, residual=r)
    for _ in range(3):
        again = mx.mxfp4_linear(x, packed, N, bias=b, activation=activation, residual=r)
        assert torch.equal(out.view(torch.int16), again.view(torch.int16)), "not reproducible"


@pytest.mark.parametrize("M,N,K", PAIRS)
@pytest.mark.parametrize("x_pad,r_pad,o_pad", [(8, 0, 1), (40, 1, 0), (0, 4, 4), (8, 8, 8), (0, 2, 6)])
def test_strides(M, N, K, x_pad, r_pad, o_pad):
    import block_scaled_mxfp4_bf16_gb300 as mx
    packed, w, x, b, r = operands(M, N, K, torch.bfloat16, True, seed=5)
    out, store = canary_out(M, N, o_pad)
    mx.mxfp4_linear(strided(x, x_pad), packed, N, bias=b, activation="gelu_tanh", residual=strided(r, r_pad), out=out)
    assert outside_untouched(out, store)
    check(out, x, w, bias=b, activation="gelu_tanh", residual=r)


@pytest.mark.parametrize("M,N,K", PAIRS)
@pytest.mark.parametrize("start,pitch", [(1, 16), (8, 16), (8, 9)])
def test_starts_inside_wider_rows(M, N, K, start, pitch):
    # columns start .. start + N of rows of N + pitch: rows off 16 bytes from the start on, or nowhere if N is whole pieces
    import block_scaled_mxfp4_bf16_gb300 as mx
    packed, w, x, b, r = operands(M, N, K, torch.bfloat16, True, seed=6)
    r1 = torch.zeros(M, N + pitch, dtype=torch.bfloat16, device="cuda")[:, start:N + start]
    r1.copy_(r)
    b1 = torch.zeros(N + 1, dtype=torch.bfloat16, device="cuda")[1:]
    b1.copy_(b)
    store = torch.full((M, N + pitch), -7.0, dtype=torch.bfloat16, device="cuda")
    out = store[:, start:N + start]
    mx.mxfp4_linear(x, packed, N, bias=b1, activation="relu", residual=r1, out=out)
    assert bool((store[:, :start] == -7).all()) and bool((store[:, N + start:] == -7).all())
    check(out, x, w, bias=b, activation="relu", residual=r)


@pytest.mark.parametrize("M,N,K", PAIRS)
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_in_place_on_the_residual(M, N, K, pad):
    import block_scaled_mxfp4_bf16_gb300 as mx
    packed, w, x, b, r = operands(M, N, K, torch.float32, True, seed=7)
    apart = mx.mxfp4_linear(x, packed, N, bias=b, activation="silu", residual=r)
    both, store = canary_out(M, N, pad)
    both.copy_(r)
    mx.mxfp4_linear(x, packed, N, bias=b, activation="silu", residual=both, out=both)
    assert outside_untouched(both, store)
    check(both, x, w, bias=b, activation="silu", residual=r)
    check(apart, x, w, bias=b, activation="silu", residual=r)
    if pad % 8 == 0:                                    # stored the same way
        assert torch.equal(both.view(torch.int16), apart.view(torch.int16))


@pytest.mark.parametrize("activation", ACTS)
@pytest.mark.parametrize("M,I,K", GATED_PAIRS)
@pytest.mark.parametrize("o_pad", [0, 3])
def test_gated(M, I, K, o_pad, activation):
    import block_scaled_mxfp4_bf16_gb300 as mx
    packed, w = gated_weights(1, I, K, seed=2)
    x = workloads.random_bf16(M, K, seed=3).cuda()
    b = 5 * random_bias(torch.float32, 4, 2 * I)
    out, store = canary_out(M, I, o_pad)
    mx.mxfp4_gated_linear(x, packed[0], I, bias=b, activation=activation, out=out)
    assert outside_untouched(out, store)
    assert mx.mxfp4_device_status() == 0
    assert_within(out, *gated(quantized(x), w[0], b, activation))
