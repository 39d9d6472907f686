"""Routing (mxfp4_moe_route) of many tokens, whose pairs are counted in chunks, against a vectorised 64-bit
definition: both types, every width of a lane's list, odd numbers of experts (two counts share a word),
masks, ties, the tail of rows that no pair takes, and the weights."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def reference(logits, k, renormalize):
    x = logits.double()
    T, E = x.shape
    key = torch.where(torch.isnan(x), -math.inf, x)
    order = torch.sort(key, dim=1, descending=True, stable=True)
    top, experts = order.values[:, :k], order.indices[:, :k]
    live = top > -math.inf
    best = top[:, :1]
    p = torch.where(key == best, 1.0, torch.exp(key - best)).masked_fill(key == -math.inf, 0.0)
    chosen = p.gather(1, experts).masked_fill(~live, 0.0)
    total = (chosen if renormalize else p).sum(1, keepdim=True)
    weights = torch.where(live, chosen / total, 0.0)
    experts = torch.where(live, experts, -1)
    flat, token = experts.flatten(), torch.arange(T * k, device=x.device) // k
    # by expert, then by token: the pairs without an expert last
    by = torch.sort(torch.where(flat < 0, E, flat), stable=True).indices
    n = int(live.sum())
    rows = torch.full((T * k,), -1, dtype=torch.int64, device=x.device)
    rows[:n] = token[by[:n]]
    slots = torch.full((T * k,), -1, dtype=torch.int64, device=x.device)
    slots[by[:n]] = torch.arange(n, device=x.device)
    counts = torch.bincount(flat[flat >= 0], minlength=E)
    offsets = torch.cat((counts.new_zeros(1), counts.cumsum(0)))
    return experts, weights, offsets, rows, slots.view(T, k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(5000, 33, 8), (5000, 255, 8), (5000, 1000, 8), (4100, 20, 9), (33000, 3, 1),
                                   (1100, 512, 32), (9000, 128, 4), (40001, 61, 6), (2000, 1024, 17)])
@pytest.mark.parametrize("kind", ["normal", "ties", "masked"])
def test_many_tokens(dtype, T, E, k, kind):
    import block_scaled_mxfp4_bf16_gb300 as mx
    assert T > 32 and T * k > 32768 and k <= E          # the form that counts in chunks
    g = torch.Generator().manual_seed(T + E)
    x = 3 * torch.randn(T, E, generator=g)
    if kind == "ties":
        x = x.round()
    if kind == "masked":      # rows that keep fewer than k experts, and rows that keep none
        x[torch.rand(T, E, generator=g) < 0.7] = -math.inf
        x[torch.rand(T, E, generator=g) < 0.05] = math.nan
        x[torch.rand(T, generator=g) < 0.1] = -math.inf
        x[T // 2] = math.inf
    x = x.to(dtype).cuda()
    for renormalize in (True, False):
        r = mx.mxfp4_moe_route(x, k, renormalize=renormalize)
        experts, weights, offsets, rows, slots = reference(x, k, renormalize)
        assert torch.equal(r.experts.long(), experts)
        assert torch.equal(r.offsets.long(), offsets)
        assert torch.equal(r.rows.long(), rows)
        assert torch.equal(r.slots.long(), slots)
        # exp within 2 ulp, a sum of up to E of them (five levels of shuffles, E / 32 in a row), a division:
        # 2^-23 each; the argument v - top rounds by 2^-24 of itself, at most 2^-24 * 104 where exp is not zero
        bound = (2 + 5 + E / 32 + 2 + 104) * 2.0 ** -23
        assert float(((r.weights.double() - weights).abs() - bound * weights).max()) <= 1e-37
