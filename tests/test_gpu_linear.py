"""mxfp4_linear against 64-bit products of the oracle's quantized values: every form of the product under it (one
K slice, the split-K reductions, tiles of more than 128 tokens, the streaming product plain and in pairs), biases,
activations, residuals, strides, alignments and values out of range."""
import pytest
import torch

from block_scaled_mxfp4_bf16_gb300 import workloads
from linear_testlib import ACT_EPS, ACTS, TINY, act64, linear
from moe_testlib import assert_within, canary_out, outside_untouched, quantized, strided, weights

pytestmark = pytest.mark.gpu

# M, N, K: for every form that the automatic plan takes on a GB300 (weight-resident unsplit and split, with two and
# three issuers; fused streaming, unsplit and split; token blocks with each reduction; wide tiles; more than one wave,
# where one group of the streaming product runs, unsplit, cut and in pairs)
SHAPES = [
    (1, 1, 8), (1, 130, 520), (3, 4096, 512), (16, 200, 1040), (17, 129, 264), (32, 300, 776), (8, 2112, 7168), (31, 77, 4096),
    (1, 9933, 2056), (4, 1, 16480), (2, 40, 16520),
    (33, 1, 8), (35, 100, 264), (34, 260, 528), (100, 36, 784), (107, 301, 800), (551, 129, 800), (33, 31, 10376),
    (37, 130, 2128), (36, 260, 1304), (5, 66, 16456), (84, 100, 9976), (51, 132, 1696), (39, 68, 776), (33, 5025, 4664),
    (33, 196, 1072), (64, 7168, 2048), (200, 4096, 512), (256, 1000, 7168), (600, 260, 1000), (1024, 512, 600),
    (33, 20071, 8), (34, 20468, 312), (1, 20228, 2248), (19, 19933, 1056), (535, 6485, 8), (700, 7300, 1544), (2048, 4160, 2040),
    (3000, 1100, 4096), (1500, 4104, 1536), (2900, 2048, 4096), (1500, 4104, 7168), (4000, 4096, 5000),
    (530, 2112, 7168), (600, 2880, 4096), (300, 8192, 4096), (512, 8200, 3584), (430, 9000, 3080), (768, 1500, 3000), (150, 14336, 4096),
    (1280, 4096, 4096),
]


def operands(M, N, K, bias, residual, seed=0):
    packed, w = weights(1, N, K, seed=N + K + seed)
    x = workloads.random_bf16(M, K, seed=M + seed)
    g = torch.Generator().manual_seed(seed + M + N)
    b = None if bias is None else torch.randn(N, generator=g).to(bias).cuda()
    r = (2 * torch.randn(M, N, generator=g)).to(torch.bfloat16).cuda() if residual else None
    return packed[0], w[0], x.cuda(), b, r


def check(out, x, w, what="", **epilogue):
    import block_scaled_mxfp4_bf16_gb300 as mx
    assert mx.mxfp4_device_status() == 0
    want, slack = linear(quantized(x), w, **epilogue)
    assert_within(out, want, slack, what)


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("bias,activation,residual", [(torch.float32, "gelu", True), (torch.bfloat16, None, True),
                                                      (None, "silu", False)])
def test_shapes(M, N, K, bias, activation, residual):
    import block_scaled_mxfp4_bf16_gb300 as mx
    packed, w, x, b, r = operands(M, N, K, bias, residual)
    out, store = canary_out(M, N, 0)
    mx.mxfp4_linear(x, packed, N, bias=b, activation=activation, residual=r, out=out)
    assert outside_untouched(out, store)
    check(out, x, w, bias=b, activation=activation, residual=r)
    again = mx.mxfp4_linear(x, packed, N, bias=b, activation=activation, residual=r)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)), "not reproducible"


@pytest.mark.parametrize("activation", ACTS)
@pytest.mark.parametrize("M,N,K", [(5, 300, 1040), (3, 4096, 512), (70, 257, 1304), (256, 4096, 512), (1500, 4104, 1536)])
def test_activations(M, N, K, activation):
    import block_scaled_mxfp4_bf16_gb300 as mx
    packed, w, x, b, _ = operands(M, N, K, torch.float32, False, seed=3)
    b = 10 * b                                          # far into both tails
    check(mx.mxfp4_linear(x, packed, N, bias=b, activation=activation), x, w, bias=b, activation=activation)
    check(mx.mxfp4_linear(x, packed, N, activation=activation), x, w, activation=activation)


@pytest.mark.parametrize("M,N,K", [(6, 203, 1040), (4, 516, 264), (40, 203, 2128), (130, 204, 520), (600, 203, 1000),
                                   (551, 132, 800), (1500, 4101, 1536), (1500, 4104, 1536), (33, 20071, 8)])
@pytest.mark.parametrize("x_pad,r_pad,o_pad", [(8, 0, 1), (40, 1, 0), (0, 4, 4), (8, 8, 8), (0, 2, 6)])
def test_strides(M, N, K, x_pad, r_pad, o_pad):
    import block_scaled_mxfp4_bf16_gb300 as mx
    packed, w, x, b, r = operands(M, N, K, torch.bfloat16, True, seed=5)
    xs, rs = strided(x, x_pad), strided(r, r_pad)
    out, store = canary_out(M, N, o_pad)
    mx.mxfp4_linear(xs, packed, N, bias=b, activation="gelu_tanh", residual=rs, out=out)
    assert outside_untouched(out, store)
    check(out, x, w, bias=b, activation="gelu_tanh", residual=r)


@pytest.mark.parametrize("M,N,K", [(2, 203, 1040), (60, 204, 1304), (600, 200, 1000), (1500, 4104, 1536)])
def test_unaligned_starts(M, N, K):
    # operands that start one element into an aligned buffer: every store and load of them is of single elements
    import block_scaled_mxfp4_bf16_gb300 as mx
    packed, w, x, b, r = operands(M, N, K, torch.bfloat16, True, seed=6)
    r1 = torch.zeros(M, N + 16, dtype=torch.bfloat16, device="cuda")[:, 1:N + 1]
    r1.copy_(r)
    b1 = torch.zeros(N + 1, dtype=torch.bfloat16, device="cuda")[1:]
    b1.copy_(b)
    store = torch.full((M, N + 16), -7.0, dtype=torch.bfloat16, device="cuda")
    out = store[:, 1:N + 1]
    mx.mxfp4_linear(x, packed, N, bias=b1, activation="relu", residual=r1, out=out)
    assert bool((store[:, 0] == -7).all()) and bool((store[:, N + 1:] == -7).all())
    check(out, x, w, bias=b, activation="relu", residual=r)


@pytest.mark.parametrize("M,N,K", [(2, 203, 1040), (1, 4096, 512), (60, 204, 1304), (600, 200, 1000), (551, 132, 800),
                                   (1500, 4104, 1536), (1500, 4101, 1536), (700, 7300, 1544)])
def test_in_place_on_the_residual(M, N, K):
    import block_scaled_mxfp4_bf16_gb300 as mx
    packed, w, x, b, r = operands(M, N, K, torch.float32, True, seed=7)
    apart = mx.mxfp4_linear(x, packed, N, bias=b, residual=r)
    stream = r.clone()
    mx.mxfp4_linear(x, packed, N, bias=b, residual=stream, out=stream)
    assert torch.equal(stream.view(torch.int16), apart.view(torch.int16))
    check(stream, x, w, bias=b, residual=r)


@pytest.mark.parametrize("M,N,K", [(8, 2112, 7168), (33, 196, 1072), (256, 1000, 7168), (600, 260, 1000)])
def test_without_an_epilogue_it_is_the_plain_product(M, N, K):
    import block_scaled_mxfp4_bf16_gb300 as mx
    packed, w, x, _, _ = operands(M, N, K, None, False)
    assert torch.equal(mx.mxfp4_linear(x, packed, N).view(torch.int16), mx.mxfp4_gemm(x, packed, N).view(torch.int16))


@pytest.mark.parametrize("M", [2, 60, 1500])
def test_infinities_and_nan_go_through_the_formula(M):
    import block_scaled_mxfp4_bf16_gb300 as mx
    N, K = 4104, 1536
    packed, w, x, b, r = operands(M, N, K, torch.float32, True, seed=8)
    b[3], b[700], b[4100] = float("inf"), float("nan"), 3.0e38
    r[0, 5], r[1, 6], r[M - 1, 4103] = float("inf"), float("nan"), float("-inf")
    for act in (None, "relu"):
        out = mx.mxfp4_linear(x, packed, N, bias=b, activation=act, residual=r).double()
        want, _ = linear(quantized(x), w, bias=b, activation=act, residual=r)
        assert torch.equal(out.isnan(), want.isnan()) and torch.equal(out.isinf(), want.float().bfloat16().isinf())
        same = want.isfinite()
        same[:, 4100] = False
        assert bool((out[same] - want[same]).abs().max() < 1.0)
    out = mx.mxfp4_linear(x, packed, N, bias=b, activation="silu").double()
    assert bool((out[:, 3] == float("inf")).all()) and bool(out[:, 700].isnan().all())
    assert int(out.isnan().sum()) == M


def test_tails_of_the_activations():
    # x = 0: the bias alone is activated, over both tails and the smallest numbers
    import block_scaled_mxfp4_bf16_gb300 as mx
    N, K = 8192, 64
    packed, _ = weights(1, N, K, seed=1)
    z = torch.cat([torch.linspace(-140, 140, N - 1024), torch.logspace(-40, 1.5, 512), -torch.logspace(-40, 1.5, 512)]).cuda()
    x = torch.zeros(1, K, dtype=torch.bfloat16, device="cuda")
    for act in ACTS:
        out = mx.mxfp4_linear(x, packed[0], N, bias=z, activation=act)[0]
        want = act64(act, z.double())
        assert_within(out[None], want[None], (want.abs() * ACT_EPS + TINY)[None], act)


@pytest.mark.parametrize("M,N,K", [(4, 300, 1040), (60, 304, 1040), (700, 7300, 1544), (700, 7304, 3080)])
def test_other_streams_graphs_and_an_empty_call(M, N, K):
    import block_scaled_mxfp4_bf16_gb300 as mx
    packed, w, x, b, r = operands(M, N, K, torch.float32, True, seed=9)
    want = mx.mxfp4_linear(x, packed, N, bias=b, residual=r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mx.mxfp4_linear(x, packed, N, bias=b, residual=r, stream=side)
    side.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    graphs, outs = [], []
    for _ in range(2):                                   # two graphs: neither shares the other's workspace
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            h = mx.mxfp4_linear(x, packed, N, bias=b, residual=r)
            outs.append(mx.mxfp4_linear(x, packed, N, bias=b, residual=h))
        graphs.append(graph)
    x2 = workloads.random_bf16(M, K, seed=77).cuda()
    x.copy_(x2)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    h = mx.mxfp4_linear(x, packed, N, bias=b, residual=r)
    want = mx.mxfp4_linear(x, packed, N, bias=b, residual=h)
    for out in outs:
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    assert mx.mxfp4_device_status() == 0
    assert mx.mxfp4_linear(x[:0], packed, N).shape == (0, N)
    assert mx.mxfp4_linear(x, packed, 0).shape == (M, 0)


@pytest.mark.parametrize("M,N,K", [(2100, 200, 520), (700, 7304, 1544), (2100, 204, 520)])
def test_rows_that_lie_past_2_to_the_31_elements(M, N, K):
    # in place, on rows far apart: the last ones start behind 2^31 elements
    import block_scaled_mxfp4_bf16_gb300 as mx
    packed, w, x, b, r = operands(M, N, K, torch.float32, True, seed=11)
    stride = (2 ** 31 + 2 ** 27) // M // 8 * 8
    store = torch.empty(M * stride, dtype=torch.bfloat16, device="cuda")
    rows = store.view(M, stride)[:, 16:16 + N]
    store.view(M, stride)[:, :N + 32] = -7.0
    rows.copy_(r)
    mx.mxfp4_linear(x, packed, N, bias=b, activation="silu", residual=rows, out=rows)
    check(rows, x, w, bias=b, activation="silu", residual=r)
    assert bool((store.view(M, stride)[:, :16] == -7).all()) and bool((store.view(M, stride)[:, 16 + N:N + 32] == -7).all())


def test_two_threads_on_one_stream():
    # calls of two kernels, enqueued with the interpreter's lock released between them
    import threading

    import block_scaled_mxfp4_bf16_gb300 as mx
    cases = [operands(300, 520, 2056, torch.float32, True, seed=s) for s in (1, 2)]
    want = [mx.mxfp4_linear(x, packed, 520, bias=b, residual=r) for packed, _, x, b, r in cases]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        packed, _, x, b, r = cases[i]
        for _ in range(200):
            got[i].append(mx.mxfp4_linear(x, packed, 520, bias=b, residual=r))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o.view(torch.int16), want[i].view(torch.int16)) for o in got[i])
    assert mx.mxfp4_device_status() == 0
