"""The grouped GEMM's pairs of CTAs (large groups) where K is just long enough for them, and tiles whose halves are an
odd number of 1 KB rows, so that a copy takes one row more than it needs."""
import pytest
import torch

from block_scaled_mxfp4_bf16_gb300 import workloads
from moe_testlib import canary_out, outside_untouched, quantized, weights
from test_gpu_grouped import check, offsets_of

pytestmark = pytest.mark.gpu


# tiles of 16, 32 .. 192 rows: every box, the last of them at the end of the token blocks
@pytest.mark.parametrize("sizes", [[600, 0, 1, 193], [16, 32, 48, 64, 900], [80, 96, 112, 128, 700, 1], [144, 160, 176, 192, 600],
                                   [400, 15], [1000, 129]])
@pytest.mark.parametrize("N,K", [(300, 1288), (640, 1536), (257, 1800)])
def test_short_k_and_every_tile_height(sizes, N, K):
    import block_scaled_mxfp4_bf16_gb300 as mx
    packed, w = weights(len(sizes), N, K, seed=N)
    a = workloads.random_bf16(sum(sizes), K, seed=K).cuda()
    c, store = canary_out(sum(sizes), N, 8)
    mx.mxfp4_grouped_gemm(a, packed, offsets_of(sizes), N, c=c)
    assert mx.mxfp4_device_status() == 0
    assert outside_untouched(c, store)
    check(c, quantized(a), w, sizes)
    again, _ = canary_out(sum(sizes), N, 8)
    mx.mxfp4_grouped_gemm(a, packed, offsets_of(sizes), N, c=again)
    assert torch.equal(c.view(torch.int16), again.view(torch.int16)), "not reproducible"
