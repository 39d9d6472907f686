"""mxfp4_linear in place: out may be the residual, but not x itself, not even where the residual is x too. One CTA would
store rows that another has yet to read and quantize. Refused before a device is asked for."""
import block_scaled_mxfp4_bf16_gb300 as mx
from test_moe_checks import ARG, P


def call(x, res, out):
    L = mx.load_library()
    return L.mxfp4_linear(x, 2, 256, 256, P + (1 << 20), 256, None, 0, 0, res, 256, out, 256, None, 0, None)


def test_out_is_not_x():
    assert call(P, None, P) == ARG
    assert call(P, P, P) == ARG
    assert call(P, P + (1 << 16), P) == ARG
