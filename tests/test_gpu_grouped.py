"""The grouped GEMM (mxfp4_grouped_gemm) against 64-bit products of the oracle's quantized values,
over ragged and empty groups, gathered rows, the gated form and operands of every stride."""
import pytest
import torch

from block_scaled_mxfp4_bf16_gb300 import workloads
from moe_testlib import assert_within, canary_out, outside_untouched, quantized, strided, sum_bound, weights

pytestmark = pytest.mark.gpu


def offsets_of(sizes, first=0):
    o = [first]
    for s in sizes:
        o.append(o[-1] + s)
    return torch.tensor(o, dtype=torch.int32, device="cuda")


def check(c, aq, w, sizes, first=0, extra=None):
    """C's group rows against aq (64 bits, one row per row of C) times each group's weights."""
    at = first
    K = aq.shape[1]
    for e, n in enumerate(sizes):
        rows = slice(at, at + n)
        if n:
            slack = aq[rows].abs() @ w[e].abs().T * sum_bound(K)
            if extra is not None:
                slack = slack + extra[rows] @ w[e].abs().T
            assert_within(c[rows], aq[rows] @ w[e].T, slack, f"group {e} of {n} rows")
        at += n


SIZES = {
    "sparse": [1, 0, 2, 0, 0, 1, 0, 3],                # few rows a group: quantized inside the product
    "one_row_each": [1] * 8,
    "ends_empty": [0, 0, 30, 17, 0, 64, 65, 0],        # 64-row tiles
    "uneven": [5, 130, 0, 1, 257, 90, 16, 400],        # 128-row tiles
    "large": [600, 0, 1000, 193, 384],                 # 192-row tiles
    "single": [77],
    "all_in_one": [0, 0, 500, 0],
}


@pytest.mark.parametrize("name", SIZES)
@pytest.mark.parametrize("N,K", [(1, 8), (128, 256), (300, 520), (129, 4096), (2048, 1024)])
@pytest.mark.parametrize("gathered", [False, True])
def test_ragged_groups(name, N, K, gathered):
    import block_scaled_mxfp4_bf16_gb300 as mx
    sizes = SIZES[name]
    R = sum(sizes)
    packed, w = weights(len(sizes), N, K, seed=N + K)
    if gathered:
        tokens = max(1, R // 3)
        a = workloads.random_bf16(tokens, K, seed=R).cuda()
        rows = torch.randint(tokens, (R,), generator=torch.Generator().manual_seed(R), dtype=torch.int32).cuda()
        aq = quantized(a)[rows.long()]
    else:
        a, rows = workloads.random_bf16(R, K, seed=R).cuda(), None
        aq = quantized(a)
    c = mx.mxfp4_grouped_gemm(a, packed, offsets_of(sizes), N, rows=rows)
    assert mx.mxfp4_device_status() == 0
    check(c, aq, w, sizes)
    again = mx.mxfp4_grouped_gemm(a, packed, offsets_of(sizes), N, rows=rows)
    assert torch.equal(c.view(torch.int16), again.view(torch.int16)), "not reproducible"


# one unit of many steps split over the SMs, long runs, and waves with a split rest
@pytest.mark.parametrize("sizes,N,K", [([100, 60], 256, 16384), ([20, 0, 20], 1000, 7168), ([700, 300], 4096, 3328),
                                       ([3, 1], 700, 8192), ([150] * 30, 640, 2048)])
def test_split_units(sizes, N, K):
    import block_scaled_mxfp4_bf16_gb300 as mx
    packed, w = weights(len(sizes), N, K, seed=7)
    a = workloads.random_bf16(sum(sizes), K, seed=1).cuda()
    c = mx.mxfp4_grouped_gemm(a, packed, offsets_of(sizes), N)
    check(c, quantized(a), w, sizes)
    for _ in range(3):
        assert torch.equal(mx.mxfp4_grouped_gemm(a, packed, offsets_of(sizes), N).view(torch.int16), c.view(torch.int16))
    assert mx.mxfp4_device_status() == 0


@pytest.mark.parametrize("E", [1, 33, 400, 1024])
def test_many_groups(E):
    import block_scaled_mxfp4_bf16_gb300 as mx
    N, K = 136, 264
    packed, w = weights(E, N, K, seed=E)
    sizes = torch.randint(0, 4, (E,), generator=torch.Generator().manual_seed(E)).tolist()
    sizes[-1] = 70
    a = workloads.random_bf16(sum(sizes), K, seed=2).cuda()
    c = mx.mxfp4_grouped_gemm(a, packed, offsets_of(sizes), N)
    check(c, quantized(a), w, sizes)
    assert mx.mxfp4_device_status() == 0


@pytest.mark.parametrize("sizes", [[1, 0, 2], [40, 0, 3], [300, 200, 0]])
@pytest.mark.parametrize("lda_pad,ldc_pad", [(8, 0), (40, 1), (8, 8)])
def test_strides_and_rows_outside_the_groups(sizes, lda_pad, ldc_pad):
    import block_scaled_mxfp4_bf16_gb300 as mx
    N, K, first, tail = 200, 328, 3, 5
    R = first + sum(sizes) + tail
    packed, w = weights(len(sizes), N, K, seed=5)
    a = strided(workloads.random_bf16(R, K, seed=4), lda_pad)
    c, store = canary_out(R, N, ldc_pad)
    mx.mxfp4_grouped_gemm(a, packed, offsets_of(sizes, first), N, c=c)
    assert mx.mxfp4_device_status() == 0
    assert outside_untouched(c, store)
    assert bool((c[:first] == -7.0).all()) and bool((c[R - tail:] == -7.0).all()), "rows of no group were written"
    check(c, quantized(a), w, sizes, first)


@pytest.mark.parametrize("sizes", [[2, 3], [40, 50]])
def test_an_index_outside_the_tokens_is_a_row_of_zeros(sizes):
    import block_scaled_mxfp4_bf16_gb300 as mx
    N, K, tokens = 150, 512, 9
    R = sum(sizes)
    packed, w = weights(2, N, K, seed=5)
    a = workloads.random_bf16(tokens, K, seed=4).cuda()
    rows = (torch.arange(R, dtype=torch.int32) % tokens).cuda()
    rows[1], rows[3], rows[R - 1] = -1, tokens, -2 ** 31
    c = mx.mxfp4_grouped_gemm(a, packed, offsets_of(sizes), N, rows=rows)
    ok = (rows >= 0) & (rows < tokens)
    assert bool((c[~ok] == 0).all())
    check(c, torch.where(ok[:, None], quantized(a)[rows.clamp(0, tokens - 1).long()], 0.0), w, sizes)


@pytest.mark.parametrize("offsets", [[0, 5, 3, 8], [0, 4, 9, 8], [-1, 2, 4, 8], [0, 2, 4, 9], [8, 4, 2, 0],
                                     [2 ** 31 - 1, -2 ** 31, 0, 8]])
@pytest.mark.parametrize("tokens", [8, 400])
def test_broken_offsets_leave_c_unwritten(offsets, tokens):
    import block_scaled_mxfp4_bf16_gb300 as mx
    N, K = 128, 256
    packed, _ = weights(3, N, K, seed=5)
    a = workloads.random_bf16(tokens, K, seed=4).cuda()
    scaled = [o if abs(o) > 100 else o * (tokens // 8) for o in offsets]
    c, store = canary_out(tokens, N, 0)
    mx.mxfp4_grouped_gemm(a, packed, torch.tensor(scaled, dtype=torch.int64).to(torch.int32).cuda(), N, c=c)
    assert mx.mxfp4_device_status() == 0
    assert bool((store == -7.0).all())


def gated_reference(a):
    """(MXFP4(silu(g) u) in 64 bits, and how far each element may be off it): the product is formed in
    fp32 within 2^-18 of its value, so an element that close to the midpoint of two e2m1 values, or a
    block whose maximum lies that close to where its scale changes, may come out on either side."""
    K = a.shape[1] // 2
    g, u = a[:, :K].double(), a[:, K:].double()
    h = torch.nn.functional.pad(g * torch.sigmoid(g) * u, (0, -K % 32)).unflatten(1, (-1, 32))
    amax = h.abs().amax(2, keepdim=True)
    mant, expo = torch.frexp(amax)
    up = mant >= 0.875
    step = torch.exp2((expo - 1 + up.int() - 2).clamp(-127, 127).double())
    v = (h / step).abs()
    spacing = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0)).double()
    q = (torch.round(v / spacing) * spacing).clamp(max=6.0)
    near = ((v / spacing - torch.floor(v / spacing) - 0.5).abs() * spacing < v * 2.0 ** -18) | (v < 2.0 ** -18)
    off = torch.where(near, spacing, 0.0) * step
    off = torch.where((mant - 0.875).abs() < 2.0 ** -18, 2 * step * spacing, off)
    value = torch.copysign(q, h) * step
    return value.flatten(1)[:, :K].contiguous(), off.flatten(1)[:, :K].contiguous()


@pytest.mark.parametrize("name", ["sparse", "ends_empty", "uneven", "large"])
@pytest.mark.parametrize("N,K", [(130, 8), (256, 520), (384, 2048)])
def test_gated(name, N, K):
    import block_scaled_mxfp4_bf16_gb300 as mx
    sizes = SIZES[name]
    R = sum(sizes)
    packed, w = weights(len(sizes), N, K, seed=N + K)
    a = workloads.random_bf16(R, 2 * K, seed=R, scale=2.0)
    a[0, :K] = -200.0          # exp overflows in fp32
    a[R - 1, K:] = 0.0         # a row of zeros
    a = strided(a, 8)
    c = mx.mxfp4_grouped_gemm(a, packed, offsets_of(sizes), N, gated=True)
    assert mx.mxfp4_device_status() == 0
    aq, off = gated_reference(a)
    assert bool((c[R - 1] == 0).all())
    check(c, aq, w, sizes, extra=off)


def test_gathered_and_gated_together():
    import block_scaled_mxfp4_bf16_gb300 as mx
    sizes, N, K, tokens = [4, 0, 9], 200, 256, 5
    packed, w = weights(3, N, K, seed=2)
    a = workloads.random_bf16(tokens, 2 * K, seed=3).cuda()
    rows = (torch.arange(13, dtype=torch.int32) * 7 % tokens).cuda()
    c = mx.mxfp4_grouped_gemm(a, packed, offsets_of(sizes), N, rows=rows, gated=True)
    aq, off = gated_reference(a)
    check(c, aq[rows.long()], w, sizes, extra=off[rows.long()])


def test_streams_graph_replays_and_a_used_workspace():
    import block_scaled_mxfp4_bf16_gb300 as mx
    N, K = 700, 8192
    for sizes in ([3, 1, 0], [90, 20, 7], [300, 0, 200]):
        packed, w = weights(3, N, K, seed=2)
        a = workloads.random_bf16(sum(sizes), K, seed=3).cuda()
        o = offsets_of(sizes)
        want = mx.mxfp4_grouped_gemm(a, packed, o, N)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(3)]
        outs = [mx.mxfp4_grouped_gemm(a, packed, o, N, stream=s) for s in streams for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(x.view(torch.int16), want.view(torch.int16)) for x in outs)
        c = torch.empty_like(want)
        ws = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(streams[0]):
            mx.mxfp4_grouped_gemm(a, packed, o, N, c=c, workspace=ws)
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=streams[0]):
                mx.mxfp4_grouped_gemm(a, packed, o, N, c=c, workspace=ws)
        for fill in (0, 255, 3):
            ws.fill_(fill)
            c.zero_()
            for _ in range(3):
                graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(c.view(torch.int16), want.view(torch.int16))
        # the graph follows the sizes it finds: other groups, same total
        o.copy_(offsets_of([sizes[2], sizes[0], sizes[1]]))
        graph.replay()
        torch.cuda.synchronize()
        check(c, quantized(a), w, [sizes[2], sizes[0], sizes[1]])
    assert mx.mxfp4_device_status() == 0


def test_empty_calls_are_no_ops():
    import block_scaled_mxfp4_bf16_gb300 as mx
    packed, _ = weights(2, 128, 256, seed=1)
    none = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    assert mx.mxfp4_grouped_gemm(none, packed, offsets_of([0, 0]), 128).shape == (0, 128)
    c, store = canary_out(4, 128, 0)
    mx.mxfp4_grouped_gemm(torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda"), packed, offsets_of([0, 0]), 128, c=c)
    torch.cuda.synchronize()
    assert bool((store == -7.0).all())


# Large groups and K of eight steps or more: two CTAs to a unit. An odd number of weight tiles, ragged N,
# groups of one row between large ones, rows outside the groups and a C whose rows are not aligned.
@pytest.mark.parametrize("sizes", [[600, 0, 1, 193, 384], [1030], [150, 129, 400, 17, 0, 0]])
@pytest.mark.parametrize("N,K,ldc_pad", [(384, 2048, 0), (300, 1800, 1), (137, 2304, 8), (1152, 2056, 2)])
def test_pairs_of_ctas(sizes, N, K, ldc_pad):
    import block_scaled_mxfp4_bf16_gb300 as mx
    first, tail = 2, 3
    R = first + sum(sizes) + tail
    packed, w = weights(len(sizes), N, K, seed=9)
    a = workloads.random_bf16(R, K, seed=3).cuda()
    c, store = canary_out(R, N, ldc_pad)
    mx.mxfp4_grouped_gemm(a, packed, offsets_of(sizes, first), N, c=c)
    assert mx.mxfp4_device_status() == 0
    assert outside_untouched(c, store)
    assert bool((c[:first] == -7.0).all()) and bool((c[R - tail:] == -7.0).all()), "rows of no group were written"
    check(c, quantized(a), w, sizes, first)
    again, _ = canary_out(R, N, ldc_pad)
    mx.mxfp4_grouped_gemm(a, packed, offsets_of(sizes, first), N, c=again)
    assert torch.equal(c.view(torch.int16), again.view(torch.int16)), "not reproducible"


@pytest.mark.parametrize("offsets", [[0, 900, 300, 800], [0, 400, 801, 800], [-1, 200, 400, 800], [800, 400, 200, 0]])
def test_broken_offsets_of_large_groups_leave_c_unwritten(offsets):
    import block_scaled_mxfp4_bf16_gb300 as mx
    N, K, tokens = 256, 2048, 800
    packed, _ = weights(3, N, K, seed=5)
    a = workloads.random_bf16(tokens, K, seed=4).cuda()
    c, store = canary_out(tokens, N, 0)
    mx.mxfp4_grouped_gemm(a, packed, torch.tensor(offsets, dtype=torch.int32).cuda(), N, c=c)
    assert mx.mxfp4_device_status() == 0
    assert bool((store == -7.0).all())


# A few units more than SMs (or pairs): the last full wave is cut into runs together with the rest, so that a
# run ends one unit, may take one whole and begins another.
@pytest.mark.parametrize("sizes,N,K", [([60] * 20, 1024, 4096), ([60] * 40, 1000, 4104), ([128, 1, 0, 127] * 11, 1025, 2816),
                                       ([300] * 10, 1100, 4096), ([190] * 20, 1024, 3584)])
def test_a_wave_cut_together_with_the_rest(sizes, N, K):
    import block_scaled_mxfp4_bf16_gb300 as mx
    packed, w = weights(len(sizes), N, K, seed=11)
    a = workloads.random_bf16(sum(sizes), K, seed=6).cuda()
    c = mx.mxfp4_grouped_gemm(a, packed, offsets_of(sizes), N)
    check(c, quantized(a), w, sizes)
    for _ in range(3):
        assert torch.equal(mx.mxfp4_grouped_gemm(a, packed, offsets_of(sizes), N).view(torch.int16), c.view(torch.int16))
    assert mx.mxfp4_device_status() == 0
