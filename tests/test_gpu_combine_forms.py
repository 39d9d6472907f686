"""Combination (mxfp4_moe_combine) in every form of its kernel: rows of 16-, 8-, 4- and 2-byte pieces, few pieces
and many, and a row that is nearly 2^31 elements long."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_a_row_of_nearly_2_to_31_elements():
    # one weight of 1: out is y's row. An odd N: single elements, so the last part of the row ends past 2^31
    import block_scaled_mxfp4_bf16_gb300 as mx
    N = (1 << 31) - 1
    if torch.cuda.get_device_properties(0).total_memory < 24 << 30:
        pytest.skip("needs 13 GB of device memory")
    bits = torch.randint(0x3C00, 0x7C00, (1, N), dtype=torch.int16, device="cuda")    # positive finite values of all kinds
    y = bits.view(torch.bfloat16)
    out = torch.empty(1, N, dtype=torch.bfloat16, device="cuda")
    mx.mxfp4_moe_combine(y, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.ones(1, 1, device="cuda"), out=out)
    assert torch.equal(out.view(torch.int16), bits)


# N, then the rows' padding: pieces of 8, 4, 2 and 1 elements on both sides of 65536 pieces, with slots past the
# eight (or four) that are in flight at once
@pytest.mark.parametrize("N,pad,vec", [(7168, 0, 8), (264, 8, 8), (2884, 0, 4), (268, 4, 4), (2882, 0, 2), (266, 2, 2),
                                       (1030, 1, 1), (2881, 0, 1)])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("k", [1, 4, 9])
def test_pieces(N, pad, vec, many, k):
    import block_scaled_mxfp4_bf16_gb300 as mx
    T = (65536 // (N // vec) + 3) if many else max(1, min(20, 65536 // (N // vec)))
    assert (T * (N // vec) > 65536) == many
    R = 3 * T + 5
    g = torch.Generator().manual_seed(N + k)
    y = torch.full((R, N + pad), 1e30, dtype=torch.bfloat16)
    y[:, :N] = torch.randn(R, N, generator=g).to(torch.bfloat16)
    slots = torch.randint(R, (T, k), generator=g, dtype=torch.int32)
    slots[torch.rand(T, k, generator=g) < 0.1] = -1
    slots[torch.rand(T, k, generator=g) < 0.05] = R          # out of range: adds nothing
    slots[T // 2] = -1                                        # nothing at all: zeros
    w = torch.randn(T, k, generator=g)
    w[slots < 0] = math.nan                                   # the weight of no row is not used
    live = (slots >= 0) & (slots < R)
    y, slots, w, live = y.cuda(), slots.cuda(), w.cuda(), live.cuda()
    want = torch.zeros(T, N, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    for j in range(k):
        term = y[:, :N][slots[:, j].clamp(0, R - 1).long()].double() * torch.where(live[:, j], w[:, j].double(), 0.0)[:, None]
        want += term
        size += term.abs()
    store = torch.full((T + 1, N + pad), -7.0, dtype=torch.bfloat16, device="cuda")
    out = store[:T, :N]
    mx.mxfp4_moe_combine(y[:, :N], slots, w, out=out)
    # k fused multiply-adds of 2^-24 each, one rounding to bf16
    err, bound = (out.double() - want).abs(), want.abs() * 2.0 ** -8 + size * (k * 2.0 ** -24) * (1 + 2.0 ** -8)
    assert bool((err <= bound).all())
    assert bool((out[T // 2] == 0).all())
    assert bool((store[T] == -7.0).all()) and bool((store[:, N:] == -7.0).all())
