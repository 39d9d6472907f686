"""The weight-only product (mxfp4_gemv) against the 64-bit product of the bf16 activations and the
values the weights stand for, within bounds derived in moe_testlib."""
import pytest
import torch

from block_scaled_mxfp4_bf16_gb300 import workloads
from moe_testlib import assert_within, canary_out, outside_untouched, strided, sum_bound, weights

pytestmark = pytest.mark.gpu


def check(x, packed, w, N, y, what=""):
    """y against x . w^T: bf16 rounding, the expansion's 2^-22 of each block's maximum, fp32 sums."""
    K = x.shape[1]
    xd = x.double()
    pad = torch.nn.functional.pad(xd.abs(), (0, -K % 32)).unflatten(1, (-1, 32))
    block_max = pad.amax(2, keepdim=True).expand_as(pad).flatten(1)[:, :K]
    want = xd @ w.T
    # the terms' magnitudes add up to at most 2 max|x| per element
    slack = block_max @ w.abs().T * (2.0 ** -22 + 2 * sum_bound(8 * K))
    assert_within(y, want, slack, what)


# each way a call is planned: one and two tokens (expanded in the product), more (a launch before),
# several token tiles; units for less than half of the SMs (clusters of 2..8), whole waves, a split
# rest; K of one to many 256-K steps and cut blocks; N below, at and past tile borders
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 8), (1, 127, 40), (1, 129, 256), (1, 4096, 512), (1, 2112, 7168), (1, 7168, 2048), (1, 20000, 1032),
    (1, 20000, 7168), (2, 640, 2040), (2, 9000, 4096), (3, 300, 264), (4, 2880, 2040), (5, 12289, 3080), (8, 2112, 7168),
    (11, 2880, 2040), (15, 64, 8192), (16, 7168, 7168), (16, 25000, 2048), (17, 200, 512), (33, 1000, 1288),
    (100, 129, 768),
])
def test_matches_64_bits(M, N, K):
    import block_scaled_mxfp4_bf16_gb300 as mx
    packed, w = weights(1, N, K, seed=N + K)
    x = workloads.random_bf16(M, K, seed=M).cuda()
    y = mx.mxfp4_gemv(x, packed[0], N)
    assert mx.mxfp4_device_status() == 0
    check(x, packed[0], w[0], N, y)
    for _ in range(3):
        assert torch.equal(mx.mxfp4_gemv(x, packed[0], N).view(torch.int16), y.view(torch.int16)), "not reproducible"


@pytest.mark.parametrize("M,ldx_pad,ldy_pad", [(1, 8, 3), (2, 24, 8), (7, 8, 1), (16, 16, 5)])
def test_strided_operands_stay_inside(M, ldx_pad, ldy_pad):
    import block_scaled_mxfp4_bf16_gb300 as mx
    N, K = 333, 1000
    packed, w = weights(1, N, K, seed=3)
    x = strided(workloads.random_bf16(M, K, seed=5), ldx_pad)
    y, store = canary_out(M, N, ldy_pad)
    mx.mxfp4_gemv(x, packed[0], N, y=y)
    assert mx.mxfp4_device_status() == 0
    assert outside_untouched(y, store)
    check(x, packed[0], w[0], N, y)


@pytest.mark.parametrize("M", [1, 6])
def test_outliers_zeros_and_small_values(M):
    import block_scaled_mxfp4_bf16_gb300 as mx
    N, K = 256, 1024
    packed, w = weights(1, N, K, seed=9)
    x = workloads.random_bf16(M, K, seed=2).float()
    x[:, ::37] *= 3000.0
    x[:, 64:96] = 0.0
    x[:, 128:160] *= 2.0 ** -100
    x[:, 160:192] *= 2.0 ** -60
    x[:, 192:224] *= 2.0 ** 90
    x = x.to(torch.bfloat16).cuda()
    y = mx.mxfp4_gemv(x, packed[0], N)
    check(x, packed[0], w[0], N, y)
    # each scale alone, so that it is not hidden by the others
    for lo in (128, 160, 192):
        z = torch.zeros_like(x)
        z[:, lo:lo + 32] = x[:, lo:lo + 32]
        check(z, packed[0], w[0], N, mx.mxfp4_gemv(z, packed[0], N), f"block at {lo}")
    assert bool((mx.mxfp4_gemv(torch.zeros_like(x), packed[0], N) == 0).all())


@pytest.mark.parametrize("M", [2, 9])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_nonfinite_token_gives_nan_and_leaves_the_others(M, bad):
    import block_scaled_mxfp4_bf16_gb300 as mx
    N, K = 300, 520
    packed, w = weights(1, N, K, seed=4)
    x = workloads.random_bf16(M, K, seed=8).cuda()
    clean = mx.mxfp4_gemv(x, packed[0], N)
    x2 = x.clone()
    x2[1, 77] = bad
    y = mx.mxfp4_gemv(x2, packed[0], N)
    assert bool(torch.isnan(y[1]).all())
    keep = [m for m in range(M) if m != 1]
    assert torch.equal(y[keep].view(torch.int16), clean[keep].view(torch.int16))


def test_no_tokens_and_no_rows_are_no_ops():
    import block_scaled_mxfp4_bf16_gb300 as mx
    packed, _ = weights(1, 128, 256, seed=1)
    assert mx.mxfp4_gemv(torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"), packed[0], 128).shape == (0, 128)
    assert mx.mxfp4_gemv(torch.zeros(2, 256, dtype=torch.bfloat16, device="cuda"), packed[0], 0).shape == (2, 0)


def test_reads_the_weights_the_gemm_reads():
    # activations that 4 bits hold exactly: both products are the same sums
    import block_scaled_mxfp4_bf16_gb300 as mx
    N, K = 384, 512
    packed, w = weights(1, N, K, seed=6)
    g = torch.Generator().manual_seed(1)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
    x = grid[torch.randint(8, (4, K), generator=g)] * torch.where(torch.rand(4, K, generator=g) < 0.5, -1.0, 1.0)
    x[:, ::32] = 4.0          # every block's maximum keeps its scale at 1
    x = x.clamp(-4.0, 4.0).to(torch.bfloat16).cuda()
    c = mx.mxfp4_gemm(x, packed[0], N)
    y = mx.mxfp4_gemv(x, packed[0], N)
    check(x, packed[0], w[0], N, y)
    assert_within(c, y.double(), x.double().abs() @ w[0].abs().T * sum_bound(K) + y.double().abs() * 2.0 ** -8, "gemm")


def test_streams_and_graph_replays():
    import block_scaled_mxfp4_bf16_gb300 as mx
    N, K = 7168, 7168
    packed, w = weights(1, N, K, seed=12)
    for M in (1, 3):
        x = workloads.random_bf16(M, K, seed=M).cuda()
        want = mx.mxfp4_gemv(x, packed[0], N)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(3)]
        outs = [mx.mxfp4_gemv(x, packed[0], N, stream=s) for s in streams for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(o.view(torch.int16), want.view(torch.int16)) for o in outs)
        s = streams[0]
        y = torch.empty_like(want)
        ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            mx.mxfp4_gemv(x, packed[0], N, y=y, workspace=ws)
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=s):
                mx.mxfp4_gemv(x, packed[0], N, y=y, workspace=ws)
        for fill in (0, 255, 1):
            ws.fill_(fill)          # whatever other calls leave in the workspace
            y.zero_()
            for _ in range(3):
                graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y.view(torch.int16), want.view(torch.int16))
    assert mx.mxfp4_device_status() == 0


def test_workspace_too_small_is_refused():
    import block_scaled_mxfp4_bf16_gb300 as mx
    packed, _ = weights(1, 256, 512, seed=1)
    x = torch.zeros(4, 512, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(mx.Mxfp4Error, match="WORKSPACE"):
        mx.mxfp4_gemv(x, packed[0], 256, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
