"""Routing and combination against 64-bit definitions, and the layer they make with the grouped
products."""
import math
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu


def route_reference(logits, k, renormalize=True):
    """experts, weights (64 bits), offsets, rows and slots from the definition, by plain loops over
    the tokens' sorted logits."""
    x = logits.double().cpu()
    T, E = x.shape
    experts = torch.full((T, k), -1, dtype=torch.int64)
    weights = torch.zeros(T, k, dtype=torch.float64)
    key = torch.where(torch.isnan(x), -math.inf, x)
    order = torch.sort(key, dim=1, descending=True, stable=True)
    for t in range(T):
        live = [e for e in order.indices[t, :k].tolist() if key[t, e] > -math.inf]
        if not live:
            continue
        top = key[t, live[0]].item()

        def p(v):
            return 1.0 if v == top else math.exp(v - top)
        over = live if renormalize else [e for e in range(E) if key[t, e] > -math.inf]
        total = sum(p(key[t, e].item()) for e in over)
        for j, e in enumerate(live):
            experts[t, j], weights[t, j] = e, p(key[t, e].item()) / total
    pairs = sorted((int(experts[t, j]), t, j) for t in range(T) for j in range(k) if experts[t, j] >= 0)
    rows = torch.full((T * k,), -1, dtype=torch.int64)
    slots = torch.full((T, k), -1, dtype=torch.int64)
    counts = torch.zeros(E, dtype=torch.int64)
    for i, (e, t, j) in enumerate(pairs):
        rows[i], slots[t, j] = t, i
        counts[e] += 1
    offsets = torch.cat((torch.zeros(1, dtype=torch.int64), counts.cumsum(0)))
    return experts, weights, offsets, rows, slots


def check_route(logits, k, renormalize=True):
    import block_scaled_mxfp4_bf16_gb300 as mx
    r = mx.mxfp4_moe_route(logits, k, renormalize=renormalize)
    experts, weights, offsets, rows, slots = route_reference(logits, k, renormalize)
    assert torch.equal(r.experts.cpu().long(), experts)
    assert torch.equal(r.offsets.cpu().long(), offsets)
    assert torch.equal(r.rows.cpu().long(), rows)
    assert torch.equal(r.slots.cpu().long(), slots)
    # exp within 2 ulp, a sum of up to E of them (five levels of shuffles, E / 32 in a row), a
    # division: 2^-23 each; the argument v - top rounds by 2^-24 of itself, at most 2^-24 * 104
    # where exp is not zero
    bound = (2 + 5 + logits.shape[1] / 32 + 2 + 104) * 2.0 ** -23
    err = (r.weights.cpu().double() - weights).abs()
    assert float((err - bound * weights).max() if err.numel() else 0.0) <= 1e-37


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (3, 5, 5), (128, 32, 4), (129, 33, 2), (200, 256, 8),
                                   (700, 100, 7), (40, 512, 16), (33, 1024, 32), (5000, 16, 2)])
@pytest.mark.parametrize("kind", ["normal", "ties", "masked"])
def test_route(dtype, T, E, k, kind):
    g = torch.Generator().manual_seed(T + E)
    x = 3 * torch.randn(T, E, generator=g)
    if kind == "ties":
        x = x.round()
    if kind == "masked":      # rows that keep fewer than k experts, and rows that keep none
        x[torch.rand(T, E, generator=g) < 0.7] = -math.inf
        x[torch.rand(T, E, generator=g) < 0.05] = math.nan
        x[T // 2] = -math.inf
    check_route(x.to(dtype).cuda(), k)
    check_route(x.to(dtype).cuda(), k, renormalize=False)


def test_route_special_logits():
    inf, nan, big = math.inf, math.nan, 3.0e38
    x = torch.tensor([[0.0, -0.0, 0.0, -0.0], [inf, 1.0, inf, -inf], [big, -big, big, nan], [nan, nan, nan, nan],
                      [-inf, -inf, -inf, 5.0], [1e-45, 0.0, -1e-45, -0.0], [-1.0, -2.0, -1.0, -2.0]])
    for dtype in (torch.float32, torch.bfloat16):
        for k in (1, 2, 4):
            check_route(x.to(dtype).cuda(), k)


@pytest.mark.parametrize("E", [2, 32, 33, 64, 200, 512, 1000])
@pytest.mark.parametrize("k", [1, 2, 8])
def test_route_takes_the_lowest_of_equal_logits(E, k):
    g = torch.Generator().manual_seed(E)
    few = torch.randint(-1, 2, (60, E), generator=g).float()
    few[:3] = 0.25            # all the same
    for dtype in (torch.float32, torch.bfloat16):
        check_route(few.to(dtype).cuda(), min(k, E))


def test_route_strided_logits_and_no_tokens():
    import block_scaled_mxfp4_bf16_gb300 as mx
    store = torch.randn(50, 100, device="cuda")
    store[:, 64:] = 1e30
    check_route(store[:, :64], 4)
    r = mx.mxfp4_moe_route(torch.empty(0, 16, device="cuda"), 4)
    assert r.offsets.tolist() == [0] * 17 and r.rows.numel() == 0 and r.experts.shape == (0, 4)


def test_route_long():
    # many chunks of tokens: the order within an expert is that of the tokens
    import block_scaled_mxfp4_bf16_gb300 as mx
    T, E, k = 40000, 64, 4
    x = torch.randn(T, E, device="cuda")
    r = mx.mxfp4_moe_route(x, k)
    top = torch.topk(x, k, dim=1).indices
    assert torch.equal(r.experts.long(), top)
    order = torch.sort(top.flatten(), stable=True).indices
    assert torch.equal(r.rows.long(), order // k)
    slots = torch.empty_like(order)
    slots[order] = torch.arange(T * k, device="cuda")
    assert torch.equal(r.slots.long(), slots.view(T, k))
    assert torch.equal(r.offsets[1:].long(), torch.bincount(top.flatten(), minlength=E).cumsum(0))


@pytest.mark.parametrize("T,k,N,R", [(1, 1, 1, 1), (5, 2, 129, 8), (64, 4, 7168, 256), (300, 8, 1000, 2400),
                                     (7, 20, 264, 140), (3, 9, 31, 5)])
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_combine(T, k, N, R, pad):
    import block_scaled_mxfp4_bf16_gb300 as mx
    g = torch.Generator().manual_seed(T * k)
    y = torch.full((R, N + pad), 1e30, dtype=torch.bfloat16)
    y[:, :N] = torch.randn(R, N, generator=g).to(torch.bfloat16)
    slots = torch.randint(R, (T, k), generator=g, dtype=torch.int32)
    slots[torch.rand(T, k, generator=g) < 0.1] = -1
    slots[torch.rand(T, k, generator=g) < 0.05] = R          # out of range: adds nothing
    slots[T - 1] = -1                                         # nothing at all: zeros
    w = torch.randn(T, k, generator=g)
    w[slots < 0] = math.nan                                   # the weight of no row is not used
    live = (slots >= 0) & (slots < R)
    rows = y[:, :N].double()[slots.clamp(0, R - 1).long()]
    wd = torch.where(live, w.double(), 0.0)[..., None]
    want, size = (rows * wd).sum(1), (rows * wd).abs().sum(1)
    store = torch.full((T + 1, N + pad), -7.0, dtype=torch.bfloat16, device="cuda")
    out = store[:T, :N]
    mx.mxfp4_moe_combine(y.cuda()[:, :N], slots.cuda(), w.cuda(), out=out)
    # k fused multiply-adds of 2^-24 each, one rounding to bf16
    err, bound = (out.cpu().double() - want).abs(), want.abs() * 2.0 ** -8 + size * (k * 2.0 ** -24) * (1 + 2.0 ** -8)
    assert bool((err <= bound).all())
    assert bool((out[T - 1] == 0).all())
    assert bool((store[T] == -7.0).all()) and bool((store[:, N:] == -7.0).all())


def test_combine_does_not_read_rows_without_a_slot():
    import block_scaled_mxfp4_bf16_gb300 as mx
    y = torch.full((4, 64), math.nan, dtype=torch.bfloat16, device="cuda")
    y[2] = 1.5
    slots = torch.tensor([[2, -1], [-1, -1], [2, 2]], dtype=torch.int32, device="cuda")
    out = mx.mxfp4_moe_combine(y, slots, torch.ones(3, 2, device="cuda"))
    assert out[:, 0].tolist() == [1.5, 0.0, 3.0]


@pytest.mark.parametrize("tokens,experts,k,hidden,intermediate", [(1, 8, 2, 512, 384), (37, 16, 4, 1024, 768),
                                                                   (300, 8, 2, 520, 264)])
def test_layer(tokens, experts, k, hidden, intermediate):
    """The example's layer. MXFP4 activations are within 1/6 of a block's maximum, about 0.1 of the
    values' norm for normal data, at each of the two products; together below 0.3."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import moe_layer

    import block_scaled_mxfp4_bf16_gb300 as mx
    g = torch.Generator("cuda").manual_seed(tokens)

    def normal(*shape, scale):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    def as_stored(w):
        # values that MXFP4 holds exactly, so that the reference's weights are the layer's
        q, s = mx.mxfp4_quantize(w.reshape(-1, w.shape[-1]))
        import oracle
        from mxfp4_testlib import to_np_u8
        v = torch.from_numpy(oracle.dequantize(to_np_u8(q), to_np_u8(s))[:, :w.shape[-1]].copy())
        return v.view(w.shape).to(torch.bfloat16).cuda()

    x = normal(tokens, hidden, scale=1.0)
    router = normal(experts, hidden, scale=hidden ** -0.5)
    w13 = as_stored(normal(experts, 2 * intermediate, hidden, scale=hidden ** -0.5))
    w2 = as_stored(normal(experts, hidden, intermediate, scale=intermediate ** -0.5))
    out = moe_layer.MoeLayer(router, w13, w2, k)(x)
    ref = moe_layer.reference(x, router, w13, w2, k)
    assert mx.mxfp4_device_status() == 0
    assert float((out.double() - ref).norm() / ref.norm()) < 0.3
