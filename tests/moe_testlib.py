"""64-bit references and error bounds for the mixture-of-experts and weight-only operators.

Bounds, none of them fitted to a result:
  * a bf16 output rounds its value by at most 2^-8 of it (eight significand bits);
  * an fp32 sum of n terms of total magnitude S is off by at most n * 2^-23 * S in any order; the
    tensor core adds 64 products at a time to the accumulator and may drop what lies below its last
    bit (2^-23 of the largest addend) in each addition, so K / 64 additions and a few more for the
    split sums, each within 2^-22 of S, bound a product's sum;
  * an activation block expanded into e2m1 terms is held to 2^-22 of its largest magnitude."""
import numpy as np
import torch

import oracle
from block_scaled_mxfp4_bf16_gb300 import workloads
from mxfp4_testlib import to_np_u8


def weights(E: int, N: int, K: int, seed: int, scale: float = 0.05):
    """E experts' weights: (packed for the device, their values in 64 bits [E, N, K] on the GPU)."""
    import block_scaled_mxfp4_bf16_gb300 as mx
    w = workloads.random_bf16(E * N, K, seed, scale)
    bq, bs = mx.mxfp4_quantize(w.cuda())
    values = oracle.dequantize(to_np_u8(bq), to_np_u8(bs))[:, :K]
    nblk = bq.shape[1] // 16
    packed = mx.mxfp4_prepack_experts(bq.view(E, N, nblk * 16), bs.view(E, N, nblk))
    return packed, torch.from_numpy(np.ascontiguousarray(values)).view(E, N, K).cuda()


def quantized(a: torch.Tensor) -> torch.Tensor:
    """MXFP4(a) by the oracle, 64 bits, [rows, K] on the GPU."""
    K = a.shape[1]
    q, s = oracle.quantize(workloads.bf16_bits(a))
    return torch.from_numpy(np.ascontiguousarray(oracle.dequantize(q, s)[:, :K])).cuda()


def strided(t: torch.Tensor, pad: int, fill: float = 1.0e30) -> torch.Tensor:
    """The same rows with `pad` elements of something else between them."""
    store = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device="cuda")
    store[:, :t.shape[1]] = t
    return store[:, :t.shape[1]]


def canary_out(rows: int, cols: int, pad: int, value: float = -7.0):
    """A [rows, cols] bf16 output inside a larger buffer filled with `value`: (output, buffer)."""
    store = torch.full((rows + 1, cols + pad), value, dtype=torch.bfloat16, device="cuda")
    return store[:rows, :cols], store


def outside_untouched(out: torch.Tensor, store: torch.Tensor, value: float = -7.0) -> bool:
    mask = torch.ones_like(store, dtype=torch.bool)
    mask[:out.shape[0], :out.shape[1]] = False
    return bool((store[mask] == value).all())


def sum_bound(K: int) -> float:
    """Relative (to the sum of magnitudes) error of a product's fp32 sum over K."""
    return (K / 64 + 64) * 2.0 ** -22


def assert_within(got: torch.Tensor, want: torch.Tensor, slack: torch.Tensor, what: str = "") -> None:
    """|got - want| <= 2^-8 |want| + slack (and bf16's smallest steps)."""
    err = (got.double() - want).abs()
    bound = want.abs() * 2.0 ** -8 + slack * (1 + 2.0 ** -8) + 2.0 ** -133
    worst = float((err / bound).max()) if err.numel() else 0.0
    assert worst <= 1.0, f"{what}: error {worst:.3g} times its bound"
