"""Combination (mxfp4_moe_combine) of a row that is nearly 2^31 elements long."""
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
