"""mxfp4_gated_linear and mxfp4_grouped_gated_linear against 64-bit products of the oracle's quantized values: every
form of the product under them, features that end inside their eights and tiles, biases, activations, strides,
ragged and empty groups, and a feed-forward block made of them."""
import numpy as np
import pytest
import torch

import oracle
from block_scaled_mxfp4_bf16_gb300 import workloads
from linear_testlib import ACTS, gated, linear, product
from moe_testlib import assert_within, canary_out, outside_untouched, quantized, strided
from mxfp4_testlib import to_np_u8

pytestmark = pytest.mark.gpu

# M, I, K over the forms of test_gpu_linear (2 I weight rows, in eights), features that end inside eights and tiles
SHAPES = [
    (1, 1, 8), (1, 65, 520), (3, 2048, 512), (16, 100, 1040), (17, 64, 264), (32, 150, 776), (8, 1056, 7168), (31, 39, 4096),
    (27, 2884, 2040), (1, 4966, 2056), (4, 1, 16480), (2, 20, 16520), (1, 2048, 7168), (2, 700, 1800),
    (33, 1, 8), (35, 50, 264), (34, 130, 528), (100, 18, 784), (107, 151, 800), (551, 65, 800), (33, 15, 10376),
    (37, 66, 2128), (36, 130, 1304), (5, 33, 16456), (84, 50, 9976), (51, 67, 1696), (39, 34, 776), (33, 2513, 4664),
    (33, 98, 1072), (64, 3584, 2048), (200, 2048, 512), (256, 500, 7168), (600, 130, 1000), (1024, 256, 600),
    (33, 10036, 8), (34, 10234, 312), (1, 10114, 2248), (19, 9967, 1056), (535, 3243, 8), (700, 3650, 1544), (2048, 2080, 2040),
    (3000, 550, 4096), (1500, 2052, 1536), (2900, 1024, 4096), (1500, 2056, 7168),
    (530, 1056, 7168), (600, 1440, 4096), (300, 4096, 4096), (512, 4100, 3584), (430, 4501, 3080), (768, 750, 3000), (150, 7168, 4096),
]


def gated_weights(E, I, K, seed, scale=0.05):
    """(packed, values in 64 bits [E, 2I, K]) of E experts."""
    import block_scaled_mxfp4_bf16_gb300 as mx
    w = workloads.random_bf16(E * 2 * I, K, seed, scale)
    bq, bs = mx.mxfp4_quantize(w.cuda())
    values = oracle.dequantize(to_np_u8(bq), to_np_u8(bs))[:, :K]
    packed = mx.mxfp4_prepack_gated_experts(bq.view(E, 2 * I, -1), bs.view(E, 2 * I, -1))
    return packed, torch.from_numpy(np.ascontiguousarray(values)).view(E, 2 * I, K).cuda()


def random_bias(dtype, seed, *shape):
    return None if dtype is None else torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("M,I,K", SHAPES)
@pytest.mark.parametrize("bias,activation", [(None, "silu"), (torch.float32, "gelu"), (torch.bfloat16, "silu")])
def test_shapes(M, I, K, bias, activation):
    import block_scaled_mxfp4_bf16_gb300 as mx
    packed, w = gated_weights(1, I, K, seed=I + K)
    x = workloads.random_bf16(M, K, seed=M).cuda()
    b = random_bias(bias, M + I, 2 * I)
    out, store = canary_out(M, I, 0)
    mx.mxfp4_gated_linear(x, packed[0], I, bias=b, activation=activation, out=out)
    assert mx.mxfp4_device_status() == 0
    assert outside_untouched(out, store)
    assert_within(out, *gated(quantized(x), w[0], b, activation))
    again = mx.mxfp4_gated_linear(x, packed[0], I, bias=b, activation=activation)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)), "not reproducible"


@pytest.mark.parametrize("activation", ACTS)
@pytest.mark.parametrize("M,I,K", [(5, 150, 1040), (3, 2048, 512), (70, 129, 1304), (256, 2048, 512), (1500, 2052, 1536)])
def test_activations(M, I, K, activation):
    import block_scaled_mxfp4_bf16_gb300 as mx
    packed, w = gated_weights(1, I, K, seed=2)
    x = workloads.random_bf16(M, K, seed=3).cuda()
    b = 5 * random_bias(torch.float32, 4, 2 * I)
    assert_within(mx.mxfp4_gated_linear(x, packed[0], I, bias=b, activation=activation),
                  *gated(quantized(x), w[0], b, activation))


@pytest.mark.parametrize("M,I,K", [(6, 103, 1040), (4, 258, 264), (40, 103, 2128), (130, 102, 520), (600, 103, 1000),
                                   (551, 68, 800), (1500, 2051, 1536), (1500, 2056, 1536), (33, 10036, 8)])
@pytest.mark.parametrize("x_pad,o_pad,start", [(8, 1, 0), (40, 0, 0), (0, 4, 0), (8, 8, 0), (0, 2, 0), (0, 16, 1)])
def test_strides(M, I, K, x_pad, o_pad, start):
    import block_scaled_mxfp4_bf16_gb300 as mx
    packed, w = gated_weights(1, I, K, seed=5)
    x = workloads.random_bf16(M, K, seed=6)
    b = random_bias(torch.bfloat16, 7, 2 * I)
    whole, store = canary_out(M, I + start, o_pad)
    out = whole[:, start:]
    mx.mxfp4_gated_linear(strided(x, x_pad), packed[0], I, bias=b, out=out)
    assert mx.mxfp4_device_status() == 0
    assert outside_untouched(whole, store) and bool((whole[:, :start] == -7.0).all())
    assert_within(out, *gated(quantized(x.cuda()), w[0], b))


def offsets_of(sizes, first=0):
    o = [first]
    for s in sizes:
        o.append(o[-1] + s)
    return torch.tensor(o, dtype=torch.int32, device="cuda")


SIZES = {
    "sparse": [1, 0, 2, 0, 0, 1, 0, 3],                # few rows a group: quantized inside the product
    "one_row_each": [1] * 8,
    "ends_empty": [0, 0, 30, 17, 0, 64, 65, 0],
    "uneven": [5, 130, 0, 1, 257, 90, 16, 400],        # 128-row tiles
    "large": [600, 0, 1000, 193, 384],                 # 192-row tiles, pairs where K allows
    "single": [77],
    "all_in_one": [0, 0, 500, 0],
}


def check_groups(out, aq, w, bias, sizes, first=0, activation="silu"):
    at = first
    for e, n in enumerate(sizes):
        if n:
            want, slack = gated(aq[at:at + n], w[e], None if bias is None else bias[e], activation)
            assert_within(out[at:at + n], want, slack, f"group {e} of {n} rows")
        at += n


@pytest.mark.parametrize("name", SIZES)
@pytest.mark.parametrize("I,K", [(1, 8), (64, 256), (150, 520), (65, 4096), (1024, 1600)])
@pytest.mark.parametrize("gathered,bias", [(False, torch.float32), (True, torch.bfloat16), (True, None)])
def test_ragged_groups(name, I, K, gathered, bias):
    import block_scaled_mxfp4_bf16_gb300 as mx
    sizes = SIZES[name]
    R, E = sum(sizes), len(sizes)
    packed, w = gated_weights(E, I, K, seed=I + K)
    b = random_bias(bias, I, E, 2 * I)
    if gathered:
        tokens = max(1, R // 3)
        a = workloads.random_bf16(tokens, K, seed=R).cuda()
        rows = torch.randint(tokens, (R,), generator=torch.Generator().manual_seed(R), dtype=torch.int32).cuda()
        aq = quantized(a)[rows.long()]
    else:
        a, rows = workloads.random_bf16(R, K, seed=R).cuda(), None
        aq = quantized(a)
    out = mx.mxfp4_grouped_gated_linear(a, packed, offsets_of(sizes), I, rows=rows, bias=b)
    assert mx.mxfp4_device_status() == 0
    check_groups(out, aq, w, b, sizes)
    again = mx.mxfp4_grouped_gated_linear(a, packed, offsets_of(sizes), I, rows=rows, bias=b)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)), "not reproducible"


@pytest.mark.parametrize("sizes,I,K", [([100, 60], 128, 16384), ([20, 0, 20], 500, 7168), ([700, 300], 2048, 3328),
                                       ([3, 1], 350, 8192), ([150] * 30, 320, 2048)])
def test_split_units(sizes, I, K):
    import block_scaled_mxfp4_bf16_gb300 as mx
    packed, w = gated_weights(len(sizes), I, K, seed=7)
    b = random_bias(torch.float32, 8, len(sizes), 2 * I)
    a = workloads.random_bf16(sum(sizes), K, seed=1).cuda()
    out = mx.mxfp4_grouped_gated_linear(a, packed, offsets_of(sizes), I, bias=b, activation="gelu_tanh")
    check_groups(out, quantized(a), w, b, sizes, activation="gelu_tanh")
    for _ in range(3):
        again = mx.mxfp4_grouped_gated_linear(a, packed, offsets_of(sizes), I, bias=b, activation="gelu_tanh")
        assert torch.equal(again.view(torch.int16), out.view(torch.int16))
    assert mx.mxfp4_device_status() == 0


@pytest.mark.parametrize("sizes", [[1, 0, 2], [40, 0, 3], [300, 200, 0]])
@pytest.mark.parametrize("a_pad,o_pad", [(8, 0), (40, 1), (8, 8)])
def test_rows_outside_the_groups_are_left_as_they_were(sizes, a_pad, o_pad):
    import block_scaled_mxfp4_bf16_gb300 as mx
    I, K, first, tail = 104, 1640, 3, 5
    R = first + sum(sizes) + tail
    packed, w = gated_weights(len(sizes), I, K, seed=5)
    a = strided(workloads.random_bf16(R, K, seed=4), a_pad)
    out, store = canary_out(R, I, o_pad)
    mx.mxfp4_grouped_gated_linear(a, packed, offsets_of(sizes, first), I, out=out)
    assert mx.mxfp4_device_status() == 0
    assert outside_untouched(out, store)
    assert bool((out[:first] == -7.0).all()) and bool((out[R - tail:] == -7.0).all())
    check_groups(out, quantized(a), w, None, sizes, first)


@pytest.mark.parametrize("sizes", [[2, 3], [40, 50], [300, 250]])
def test_an_index_outside_the_tokens_is_a_row_of_zeros(sizes):
    # so its result is that of the biases alone
    import block_scaled_mxfp4_bf16_gb300 as mx
    I, K, tokens = 75, 1544, 9
    R = sum(sizes)
    packed, w = gated_weights(2, I, K, seed=5)
    b = random_bias(torch.float32, 6, 2, 2 * I)
    a = workloads.random_bf16(tokens, K, seed=4).cuda()
    rows = (torch.arange(R, dtype=torch.int32) % tokens).cuda()
    rows[1], rows[3], rows[R - 1] = -1, tokens, -2 ** 31
    out = mx.mxfp4_grouped_gated_linear(a, packed, offsets_of(sizes), I, rows=rows, bias=b)
    ok = (rows >= 0) & (rows < tokens)
    aq = torch.where(ok[:, None], quantized(a)[rows.long().clamp(0, tokens - 1)], 0.0)
    check_groups(out, aq, w, b, sizes)


@pytest.mark.parametrize("bad", [[0, 3, 2, 6], [0, 2, 4, 7], [-1, 2, 4, 6]])
@pytest.mark.parametrize("times", [1, 100])
def test_offsets_that_break_their_rule_leave_the_output(bad, times):
    import block_scaled_mxfp4_bf16_gb300 as mx
    I, K, R = 100, 1544, 6 * times
    packed, _ = gated_weights(3, I, K, seed=5)
    a = workloads.random_bf16(R, K, seed=4).cuda()
    offsets = torch.tensor([o * times for o in bad], dtype=torch.int32, device="cuda")
    out = torch.full((R, I), -7.0, dtype=torch.bfloat16, device="cuda")
    mx.mxfp4_grouped_gated_linear(a, packed, offsets, I, out=out)
    assert mx.mxfp4_device_status() == 0
    assert bool((out == -7.0).all())


@pytest.mark.parametrize("tokens", [1, 20, 700])
def test_a_feed_forward_block(tokens):
    """norm'd x -> gated product -> second product back onto the residual stream, in place, captured and replayed."""
    import block_scaled_mxfp4_bf16_gb300 as mx
    H, I = 1024, 1360
    packed, w13 = gated_weights(1, I, H, seed=1)
    w2 = workloads.random_bf16(H, I, seed=2, scale=0.05).cuda()
    q2, s2 = mx.mxfp4_quantize(w2)
    packed2 = mx.mxfp4_prepack_b(q2, s2)
    v2 = torch.from_numpy(np.ascontiguousarray(oracle.dequantize(to_np_u8(q2), to_np_u8(s2))[:, :I])).cuda()
    x = workloads.random_bf16(tokens, H, seed=3).cuda()
    residual = workloads.random_bf16(tokens, H, seed=4).cuda()
    before = residual.clone()
    b2 = random_bias(torch.float32, 5, H)

    def block():
        h = mx.mxfp4_gated_linear(x, packed[0], I)
        mx.mxfp4_linear(h, packed2, H, bias=b2, residual=residual, out=residual)
        return h
    h = block()
    assert mx.mxfp4_device_status() == 0
    assert_within(h, *gated(quantized(x), w13[0]))
    assert_within(residual, *linear(quantized(h), v2, bias=b2, residual=before))
    eager = residual.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block()
    residual.copy_(before)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(residual.view(torch.int16), eager.view(torch.int16))


@pytest.mark.parametrize("tokens", [1, 33, 900])
def test_a_mixture_of_experts_layer(tokens):
    """route -> the experts' gated products -> their second products -> combine."""
    import block_scaled_mxfp4_bf16_gb300 as mx
    from moe_testlib import weights
    E, k, H, I = 6, 2, 512, 328
    packed, w13 = gated_weights(E, I, H, seed=1)
    packed2, w2 = weights(E, H, I, seed=2)
    b = random_bias(torch.bfloat16, 3, E, 2 * I)
    x = workloads.random_bf16(tokens, H, seed=4).cuda()
    logits = torch.randn(tokens, E, generator=torch.Generator().manual_seed(5)).cuda()
    r = mx.mxfp4_moe_route(logits, k)
    h = mx.mxfp4_grouped_gated_linear(x, packed, r.offsets, I, rows=r.rows, bias=b)
    y = mx.mxfp4_grouped_gemm(h, packed2, r.offsets, H)
    out = mx.mxfp4_moe_combine(y, r.slots, r.weights)
    assert mx.mxfp4_device_status() == 0
    sizes = (r.offsets[1:] - r.offsets[:-1]).tolist()
    check_groups(h, quantized(x)[r.rows.long()], w13, b, sizes)
    hq, want = quantized(h), torch.zeros(tokens, H, dtype=torch.float64, device="cuda")
    at = 0
    yq = torch.zeros(sum(sizes), H, dtype=torch.float64, device="cuda")
    ys = torch.zeros_like(yq)
    for e, n in enumerate(sizes):
        yq[at:at + n], ys[at:at + n] = product(hq[at:at + n], w2[e])
        at += n
    ys += yq.abs() * 2.0 ** -8 * (1 + 2.0 ** -8)         # y rounds to bf16, the sum of two terms twice in fp32
    slack = torch.zeros_like(want)
    for j in range(k):
        weight, slot = r.weights[:, j, None].double(), r.slots[:, j].long()
        want += weight * yq[slot]
        slack += weight * (ys[slot] + yq[slot].abs() * 2.0 ** -22)
    assert_within(out, want, slack)


@pytest.mark.parametrize("M", [4, 700])
def test_streams_and_empty_calls(M):
    import block_scaled_mxfp4_bf16_gb300 as mx
    I, K = 3650, 1544
    packed, w = gated_weights(1, I, K, seed=1)
    x = workloads.random_bf16(M, K, seed=2).cuda()
    want = mx.mxfp4_gated_linear(x, packed[0], I)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mx.mxfp4_gated_linear(x, packed[0], I, stream=side)
    grouped = mx.mxfp4_grouped_gated_linear(x, packed, offsets_of([M]), I, stream=side)
    side.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    assert_within(grouped, *gated(quantized(x), w[0]))
    assert mx.mxfp4_gated_linear(x[:0], packed[0], I).shape == (0, I)
    assert mx.mxfp4_grouped_gated_linear(x[:0], packed, offsets_of([0]), I).shape == (0, I)
    assert mx.mxfp4_device_status() == 0
