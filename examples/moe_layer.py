"""A mixture-of-experts feed-forward layer on MXFP4 weights, the way a model's layer uses the
operators: route, the experts' first products (gate and up), the gated second products, combine.

    python examples/moe_layer.py [tokens] [experts] [k] [hidden] [intermediate]

Prints the largest deviation from the same layer computed in 64 bits from the quantized weights
(the activations are quantized to MXFP4 inside the products, so the deviation is that of 4-bit
activations), and the time of a layer."""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_mxfp4_bf16_gb300 as mx  # noqa: E402


class MoeLayer:
    """router [E, hidden] bf16; w13 [E, 2 * intermediate, hidden] and w2 [E, hidden, intermediate]
    bf16, quantized and packed here once."""

    def __init__(self, router: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor, k: int):
        self.router, self.k = router, k
        self.hidden, self.intermediate = w2.shape[1], w2.shape[2]
        self.w13 = self._pack(w13)
        self.w2 = self._pack(w2)

    @staticmethod
    def _pack(w: torch.Tensor) -> torch.Tensor:
        E, N, K = w.shape
        bq, bs = mx.mxfp4_quantize(w.reshape(E * N, K))
        return mx.mxfp4_prepack_experts(bq.view(E, N, -1), bs.view(E, N, -1))

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        r = mx.mxfp4_moe_route((x @ self.router.T).float(), self.k)
        gate_up = mx.mxfp4_grouped_gemm(x, self.w13, r.offsets, 2 * self.intermediate, rows=r.rows)
        y = mx.mxfp4_grouped_gemm(gate_up, self.w2, r.offsets, self.hidden, gated=True)
        return mx.mxfp4_moe_combine(y, r.slots, r.weights)


def reference(x: torch.Tensor, router: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor, k: int) -> torch.Tensor:
    """The layer in 64 bits on the given (dequantized) weights, activations not quantized."""
    logits = (x @ router.T).double()
    top = torch.sort(logits, dim=1, descending=True, stable=True)
    weights = torch.softmax(top.values[:, :k], 1)
    out = torch.zeros(x.shape[0], w2.shape[1], dtype=torch.float64, device=x.device)
    for j in range(k):
        for e in top.indices[:, j].unique().tolist():
            t = (top.indices[:, j] == e).nonzero().flatten()
            gate, up = (x[t].double() @ w13[e].double().T).chunk(2, 1)
            out[t] += weights[t, j, None] * ((gate * torch.sigmoid(gate) * up) @ w2[e].double().T)
    return out


def main(tokens: int = 64, experts: int = 16, k: int = 4, hidden: int = 1024, intermediate: int = 768) -> float:
    g = torch.Generator("cuda").manual_seed(0)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    x = normal(tokens, hidden)
    router = normal(experts, hidden, scale=hidden ** -0.5)
    w13 = normal(experts, 2 * intermediate, hidden, scale=hidden ** -0.5)
    w2 = normal(experts, hidden, intermediate, scale=intermediate ** -0.5)
    layer = MoeLayer(router, w13, w2, k)
    out = layer(x)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(20):
        layer(x)
    end.record()
    torch.cuda.synchronize()
    if mx.mxfp4_device_status() != 0:
        raise RuntimeError("a bounded wait ran out")
    ref = reference(x, router, w13, w2, k)
    deviation = float((out.double() - ref).norm() / ref.norm())
    print(f"{tokens} tokens, {k} of {experts} experts, {hidden} x {intermediate}: "
          f"deviation from 64 bits without quantization {deviation:.3f} (relative, 2-norm), "
          f"{start.elapsed_time(end) / 20 * 1e3:.1f} us a layer")
    return deviation


if __name__ == "__main__":
    main(*(int(v) for v in sys.argv[1:]))
