"""The linear epilogue of the streaming products waits for the pieces of the residual that its tensor copies bring. A
warp whose wait runs out says so to the whole CTA, as every other bounded wait does: the kernel ends, the status says so,
and the next call on the same workspace gives the right result (the test build's hook: see test_gpu_give_up)."""
import ctypes
import glob
import os
import re

import pytest
import torch

from block_scaled_mxfp4_bf16_gb300 import workloads

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_mxfp4_bf16_gb300", "csrc")
TIMEOUT = 6
PIECES = 1 << 20          # where the hook's numbers of these waits begin


def test_a_streaming_product_gives_up_in_one_way_only():
    # stream_fail alone writes the status, and it raises the CTA's flag with it
    writes = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*stream*"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        writes += [(os.path.basename(path), text[m.start() - 150:m.end() + 60]) for m in re.finditer(r"p\.status\b", text)]
    assert len(writes) == 1 and writes[0][0] == "stream_device.cuh", [w[0] for w in writes]
    assert re.search(r"void stream_fail\(.*atomicOr\(p\.status, 1u\);\s*\*abort_flag = 1u;", writes[0][1], re.S)


@pytest.fixture(scope="module")
def hooks():
    from block_scaled_mxfp4_bf16_gb300 import build
    L = ctypes.CDLL(build.build_variant("hooks", ["-DMXFP4_TEST_HOOKS"]))
    vp, i64, sz, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
    L.mxfp4_test_stream_give_up.argtypes = [i32, i32, i32]
    L.mxfp4_test_stream_give_up.restype = None
    L.mxfp4_linear.argtypes = [vp, i64, i64, i64, vp, i64, vp, i32, i32, vp, i64, vp, i64, vp, sz, vp]
    L.mxfp4_device_status.argtypes = [vp]
    L.mxfp4_linear_workspace_size.restype = sz
    L.mxfp4_linear_workspace_size.argtypes = [i64] * 3
    yield L
    L.mxfp4_test_stream_give_up(-1, 0, 0)


# M, N, K of several waves of whole units, CTAs alone and in pairs; CTA, thread of its epilogue (128 .. 383) and piece:
# a unit's first and last ones, pieces asked for ahead of them or not, either CTA of a pair
@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,cta,thread,piece", [
    (3648, 4096, 1536, 5, 128, 0), (3648, 4096, 1536, 151, 383, 4), (3648, 4096, 1536, 0, 255, 9),
    (8192, 4096, 7168, 3, 130, 0), (8192, 4096, 7168, 8, 300, 1), (8192, 4096, 7168, 75, 383, 13),
])
def test_a_residual_that_does_not_arrive_ends_the_kernel(hooks, M, N, K, cta, thread, piece):
    import block_scaled_mxfp4_bf16_gb300 as mx
    from moe_testlib import weights
    st = torch.cuda.current_stream().cuda_stream
    x = workloads.random_bf16(M, K, seed=4).cuda()
    r = workloads.random_bf16(M, N, seed=5).cuda()
    packed = weights(1, N, K, seed=3)[0][0]
    want = mx.mxfp4_linear(x, packed, N, activation="gelu_tanh", residual=r)
    ws = torch.full((hooks.mxfp4_linear_workspace_size(M, N, K),), 0xEE, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(want)

    def call():
        return hooks.mxfp4_linear(x.data_ptr(), M, K, K, packed.data_ptr(), N, None, 0, 4, r.data_ptr(), N, out.data_ptr(), N,
                                  ws.data_ptr(), ws.nbytes, st)
    assert hooks.mxfp4_device_status(None) == 0
    hooks.mxfp4_test_stream_give_up(cta, thread, PIECES + piece)
    assert call() == 0
    torch.cuda.synchronize()
    assert hooks.mxfp4_device_status(None) == TIMEOUT
    hooks.mxfp4_test_stream_give_up(-1, 0, 0)
    for _ in range(2):
        out.zero_()
        assert call() == 0
        torch.cuda.synchronize()
        assert hooks.mxfp4_device_status(None) == 0
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
