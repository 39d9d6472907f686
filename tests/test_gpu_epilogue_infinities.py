"""Infinities, NaN and numbers near the largest in biases and residuals go through the formula of their own element and
touch no other: every form of the products with an epilogue, every activation, finite elements held to the same bounds
as without them."""
import pytest
import torch

from block_scaled_mxfp4_bf16_gb300 import workloads
from linear_testlib import ACTS, activated, linear, product
from moe_testlib import assert_within, quantized, weights
from test_gpu_gated_linear import gated_weights, offsets_of, random_bias

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def compare(out, want, slack, sure=None, what=""):
    """NaN and infinities where the formula has them, of the same sign, and every other element within its bound."""
    got = out.double()
    sure = torch.ones_like(want, dtype=torch.bool) if sure is None else sure
    rounded = want.float().bfloat16().double()
    assert torch.equal(got.isnan() & sure, want.isnan() & sure), what
    assert torch.equal(torch.where(got.isinf() & sure, got, 0.0), torch.where(rounded.isinf() & sure, rounded, 0.0)), what
    finite = want.isfinite() & rounded.isfinite() & sure
    assert bool(finite.any())
    assert_within(got[finite], want[finite], slack[finite], what)


# a few tokens with one K slice and with split ones, token blocks with and without a split, the streaming product alone and
# in pairs, each with rows that are 16-byte aligned and not
SHAPES = [(3, 4096, 512), (16, 4100, 512), (2, 4104, 1536), (31, 77, 4096), (60, 4104, 1536), (33, 1030, 4664), (256, 1000, 7168),
          (551, 129, 800), (1500, 4104, 1536), (1500, 4101, 1536), (1500, 4104, 7168), (1500, 4101, 7168)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(M, N, K):
    import block_scaled_mxfp4_bf16_gb300 as mx
    packed, w = weights(1, N, K, seed=N + K)
    x = workloads.random_bf16(M, K, seed=M).cuda()
    g = torch.Generator().manual_seed(1)
    b = torch.randn(N, generator=g).cuda()
    r = torch.randn(M, N, generator=g).to(torch.bfloat16).cuda()
    for n, v in ((3, INF), (8, -INF), (15, NAN), (16, 3.0e38), (33, -3.0e38), (N - 2, INF)):
        b[n] = v
    r[0, 5], r[M // 2, 6], r[M - 1, N - 1], r[M - 1, 3], r[0, 40] = INF, NAN, -INF, -INF, 3.0e38
    xq = quantized(x)
    for act in ACTS:
        for residual in (None, r):
            out = mx.mxfp4_linear(x, packed[0], N, bias=b, activation=act, residual=residual)
            compare(out, *linear(xq, w[0], b, act, residual), what=f"{act} {residual is not None}")
    assert mx.mxfp4_device_status() == 0


def gated_parts(xq, w, bias, activation):
    """(value, bound, where the signs and zeros of both factors are sure) of a gated product."""
    z, slack = product(xq, w)
    I = w.shape[0] // 2
    g, gs = activated(activation, z[:, :I], slack[:, :I], bias[:I])
    u, us = activated(None, z[:, I:], slack[:, I:], bias[I:])
    out = g * u
    clear = (g.isnan() | (g.abs() > 2 * gs) | (g.abs() == INF)) & (u.isnan() | (u.abs() > 2 * us) | (u.abs() == INF))
    # relu's zero is exact where the gate is below zero by more than its bound
    if activation == "relu":
        pre = z[:, :I] + bias[:I].double()
        clear |= (pre < -2 * slack[:, :I] - pre.abs() * 2.0 ** -23) & (u.isnan() | (u.abs() > 2 * us) | (u.abs() == INF))
    special = ~(g.isfinite() & u.isfinite()) | ~out.float().bfloat16().isfinite()
    return out, gs * u.abs() + us * g.abs() + gs * us + out.abs() * 2.0 ** -24, clear | ~special


def spoiled(bias):
    """A bias [.., 2I] with infinities, NaN and large numbers in gate and up projection."""
    I = bias.shape[-1] // 2
    for n, v in ((3, INF), (8, -INF), (14, NAN), (16, 1.0e30), (I - 2, INF), (I + 5, INF), (I + 9, -INF), (I + 15, NAN), (I + 17, 3.0e36),
                 (2 * I - 1, NAN)):
        bias[..., n] = v
    return bias


GATED = [(M, N // 2, K) for M, N, K in SHAPES if N > 128] + [(40, 50, 9976), (1500, 2056, 1536), (1500, 2056, 7168)]


@pytest.mark.parametrize("M,I,K", GATED)
def test_gated(M, I, K):
    import block_scaled_mxfp4_bf16_gb300 as mx
    packed, w = gated_weights(1, I, K, seed=I + K)
    x = workloads.random_bf16(M, K, seed=M).cuda()
    b = spoiled(random_bias(torch.float32, 3, 2 * I))
    xq = quantized(x)
    for act in ACTS:
        out = mx.mxfp4_gated_linear(x, packed[0], I, bias=b, activation=act)
        compare(out, *gated_parts(xq, w[0], b, act), what=act)
    assert mx.mxfp4_device_status() == 0


@pytest.mark.parametrize("sizes", [[1, 0, 2, 3], [5, 130, 0, 257], [600, 193, 0, 384]])
@pytest.mark.parametrize("I,K", [(136, 1640), (350, 4096), (1024, 1600)])
def test_experts(sizes, I, K):
    import block_scaled_mxfp4_bf16_gb300 as mx
    E = len(sizes)
    packed, w = gated_weights(E, I, K, seed=I + K)
    a = workloads.random_bf16(sum(sizes), K, seed=2).cuda()
    b = random_bias(torch.float32, 4, E, 2 * I)
    spoiled(b[1])
    spoiled(b[3])
    xq = quantized(a)
    for act in ACTS:
        out = mx.mxfp4_grouped_gated_linear(a, packed, offsets_of(sizes), I, bias=b, activation=act)
        at = 0
        for e, n in enumerate(sizes):
            if n:
                compare(out[at:at + n], *gated_parts(xq[at:at + n], w[e], b[e], act), what=f"{act}, expert {e}")
            at += n
    assert mx.mxfp4_device_status() == 0
