"""Packed weights are one run of bytes from the buffer's start, and the kernels read it as that: a view with as many
bytes but strides of its own (an expanded byte, every other one) is refused, by every product that reads them."""
import pytest
import torch

import block_scaled_mxfp4_bf16_gb300 as mx
from test_binding_checks import dev
from test_linear_checks import bf16, gated_packed, lib, packed, ws  # noqa: F401  (lib: the fixture)


def views(good: torch.Tensor):
    """The same number of bytes, or more, that do not lie next to each other."""
    n = good.nbytes
    return (dev(torch.zeros(1, dtype=torch.uint8).expand(n)), dev(torch.zeros(2 * n, dtype=torch.uint8)[::2]),
            dev(torch.zeros(1024, n // 1024, dtype=torch.uint8).T))


CALLS = {
    "linear": lambda b: mx.mxfp4_linear(bf16(2, 256), b, 128, out=bf16(2, 128), workspace=ws(), stream=0),
    "gemv": lambda b: mx.mxfp4_gemv(bf16(2, 256), b, 128, y=bf16(2, 128), workspace=ws(), stream=0),
    "gemm": lambda b: mx.mxfp4_gemm(bf16(2, 256), b, 128, c=bf16(2, 128), workspace=ws(), stream=0),
    "gemm_noalloc": lambda b: mx.mxfp4_gemm_noalloc(bf16(2, 256), b, 128, c=bf16(2, 128), stream=0),
    "gated": lambda b: mx.mxfp4_gated_linear(bf16(2, 256), b, 64, out=bf16(2, 64), workspace=ws(), stream=0),
}


@pytest.mark.parametrize("name", CALLS)
def test_scattered_bytes_are_refused(lib, name):  # noqa: F811
    good = gated_packed(1, 64, 256)[0] if name == "gated" else packed(1, 128, 256)[0]
    CALLS[name](good)
    calls = len(lib.calls)
    for bad in views(good):
        assert bad.nbytes >= good.nbytes
        with pytest.raises(ValueError):
            CALLS[name](bad)
    assert len(lib.calls) == calls
