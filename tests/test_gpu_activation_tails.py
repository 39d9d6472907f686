"""The activations over both tails, by the bound the header states: 2^-15 of the value wherever the factor that multiplies
z is a normal number of fp32, and 2^-119 beside that only where it is not."""
import pytest
import torch

from linear_testlib import ACT_EPS, ACTS, TINY, act64
from moe_testlib import assert_within, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("activation", ACTS)
@pytest.mark.parametrize("M", [1, 40])
def test_two_to_the_minus_119_only_below_the_normal_numbers(M, activation):
    import block_scaled_mxfp4_bf16_gb300 as mx
    N, K = 8192, 64
    packed, _ = weights(1, N, K, seed=1)
    z = torch.cat([torch.linspace(-140, 140, N - 2048), -torch.linspace(87, 93, 512), -torch.linspace(9.9, 13.6, 512),
                   torch.logspace(-37, 2, 512), -torch.logspace(-37, 2, 512)]).cuda()
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    out = mx.mxfp4_linear(x, packed[0], N, bias=z, activation=activation)
    want = act64(activation, z.double())
    # twice the smallest normal number: a factor rounds, and gelu's lies within 2^-15 of its value
    small = (want / z.double()).abs() < 2.0 ** -125
    slack = want.abs() * ACT_EPS + torch.where(small, TINY, 0.0)
    assert_within(out, want.expand(M, N), slack.expand(M, N), activation)
