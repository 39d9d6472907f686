"""64-bit references and error bounds of the products with an epilogue.

Bounds, none of them fitted to a result:
  * z is a product's fp32 sum (moe_testlib.sum_bound of the sum of magnitudes), and the bias adds a rounding of
    2^-24 of what it gives;
  * no activation's slope exceeds 1.13 (gelu's maximum, 1.1290; silu 1.0998; gelu_tanh 1.1290), so that much of z's
    error passes through;
  * an activation is computed to 2^-15 of its value: the exponential's argument is below 128 in magnitude
    wherever the result is a normal number and carries at most five roundings of 2^-24 (ln 2 * 128 * 5 * 2^-24 =
    2^-15.2 of the exponential; silu one rounding), the hardware's 2^x and 1 / x 2^-22 each, gelu's fit 1.1e-5
    with two roundings of such an argument; a factor below the smallest normal number, 2^-126, counts as zero, which
    silu meets first, below z = -87.3: the result it loses is at most 88 * 2^-126 < 2^-119;
  * the product of a gated pair and the sum with a residual round once each in fp32 (2^-24);
  * the result rounds to bf16: 2^-8 of it."""
import torch

from moe_testlib import sum_bound

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
SLOPE, ACT_EPS, TINY = 1.13, 2.0 ** -15, 2.0 ** -119


def act64(name, z):
    if name in (None, "none"):
        return z
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * torch.special.erfc(-z / 2 ** 0.5) / 2   # Phi without a difference of near values
    return z * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3))


def product(xq, w):
    """(z, the bound of its fp32 sum) of xq [M, K] . w [N, K]^T."""
    return xq @ w.T, xq.abs() @ w.abs().T * sum_bound(xq.shape[1])


def activated(name, z, slack, bias):
    """(act(z + bias), its bound)."""
    if bias is not None:
        z = z + bias.double()
        slack = slack + z.abs() * 2.0 ** -24
    a = act64(name, z)
    return a, (slack if name in (None, "none") else SLOPE * slack + a.abs() * ACT_EPS + TINY)


def linear(xq, w, bias=None, activation=None, residual=None):
    a, slack = activated(activation, *product(xq, w), bias)
    if residual is not None:
        a = a + residual.double()
        slack = slack + a.abs() * 2.0 ** -24
    return a, slack


def gated(xq, w, bias=None, activation="silu"):
    """w: [2I, K], the gate's rows first."""
    z, slack = product(xq, w)
    I = w.shape[0] // 2
    g, gs = activated(activation, z[:, :I], slack[:, :I], None if bias is None else bias[:I])
    u, us = activated(None, z[:, I:], slack[:, I:], None if bias is None else bias[I:])
    out = g * u
    return out, gs * u.abs() + us * g.abs() + gs * us + out.abs() * 2.0 ** -24
