"""Streaming products in which one thread's bounded wait counts as run out: the kernel ends all the same, the
status says so, and the next call on the same workspace gives the right result. The warps of a CTA meet at
barriers, so what one thread finds has to become a decision of all of them.

A test build of the library (-DMXFP4_TEST_HOOKS, its own .so; the product library has no such hook) lets one
thread of one CTA take its warp's nth wait for run out; nothing is made to wait for something that does not
come but for the second or so that the kernel's other warps then allow."""
import ctypes

import pytest
import torch

from block_scaled_mxfp4_bf16_gb300 import workloads
from moe_testlib import weights

pytestmark = pytest.mark.gpu
TIMEOUT = 6


@pytest.fixture(scope="module")
def hooks():
    from block_scaled_mxfp4_bf16_gb300 import build
    L = ctypes.CDLL(build.build_variant("hooks", ["-DMXFP4_TEST_HOOKS"]))
    vp, i64, sz, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
    L.mxfp4_test_stream_give_up.argtypes = [i32, i32, i32]
    L.mxfp4_test_stream_give_up.restype = None
    L.mxfp4_test_stream_tag.argtypes = [ctypes.c_uint64]
    L.mxfp4_test_stream_tag.restype = None
    L.mxfp4_gemv.argtypes = [vp, i64, i64, i64, vp, i64, vp, i64, vp, sz, vp]
    L.mxfp4_grouped_gemm.argtypes = [vp, i64, i64, i64, vp, vp, i64, vp, i64, vp, i64, i64, ctypes.c_uint, vp, sz, vp]
    L.mxfp4_device_status.argtypes = [vp]
    for name in ("mxfp4_gemv_workspace_size", "mxfp4_grouped_gemm_workspace_size"):
        getattr(L, name).restype = sz
    L.mxfp4_gemv_workspace_size.argtypes = [i64] * 3
    L.mxfp4_grouped_gemm_workspace_size.argtypes = [i64] * 4
    yield L
    L.mxfp4_test_stream_give_up(-1, 0, 0)
    L.mxfp4_test_stream_tag(0)


def prepared(hooks, sizes, N, K):
    """(a call of the test build on fixed buffers, its output, the product library's output). sizes an
    int: the weight-only product of that many tokens, else a grouped product."""
    import block_scaled_mxfp4_bf16_gb300 as mx
    st = torch.cuda.current_stream().cuda_stream
    if isinstance(sizes, int):
        packed, _ = weights(1, N, K, seed=3)
        x = workloads.random_bf16(sizes, K, seed=4).cuda()
        want = mx.mxfp4_gemv(x, packed[0], N)
        ws = torch.full((hooks.mxfp4_gemv_workspace_size(sizes, N, K),), 0xEE, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(want)

        def call():
            return hooks.mxfp4_gemv(x.data_ptr(), sizes, K, K, packed.data_ptr(), N, out.data_ptr(), N, ws.data_ptr(),
                                    ws.nbytes, st)
    else:
        E, R = len(sizes), sum(sizes)
        packed, _ = weights(E, N, K, seed=3)
        a = workloads.random_bf16(R, K, seed=4).cuda()
        offsets = torch.tensor([0] + sizes).cumsum(0).int().cuda()
        want = mx.mxfp4_grouped_gemm(a, packed, offsets, N)
        ws = torch.full((hooks.mxfp4_grouped_gemm_workspace_size(R, E, N, K),), 0xEE, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(want)

        def call():
            return hooks.mxfp4_grouped_gemm(a.data_ptr(), R, K, K, None, offsets.data_ptr(), E, packed.data_ptr(), N,
                                            out.data_ptr(), R, N, 0, ws.data_ptr(), ws.nbytes, st)
    return call, out, want


# sizes, N, K, then the thread: CTA, thread, nth wait of its warp. Threads of one epilogue warp (128 .. 383):
# in a unit split among six CTAs, in runs that end one unit and begin another, in a whole unit before
# split ones, in either CTA of a pair; the weight-only product split and in clusters. Then a warp that
# writes tokens (64 .. 127) and one that writes scale factors (384 .. 639 of a pair).
CASES = [
    ([100, 60], 256, 16384, 0, 200, 0), ([100, 60], 256, 16384, 3, 130, 0), ([60] * 20, 1024, 4096, 5, 383, 0),
    ([60] * 20, 1024, 4096, 5, 255, 1), ([700, 300], 4096, 3328, 7, 140, 0), ([300] * 10, 1100, 4096, 1, 133, 0),
    ([300] * 10, 1100, 4096, 4, 300, 1), (1, 20000, 7168, 2, 170, 0), (16, 23301, 5040, 9, 190, 0),
    (1, 2112, 7168, 3, 180, 0), ([1] * 8, 4096, 4096, 6, 70, 12), ([300] * 10, 1100, 4096, 3, 400, 2),
]


@pytest.mark.parametrize("sizes,N,K,cta,thread,nth", CASES)
def test_a_wait_that_runs_out_ends_the_kernel(hooks, sizes, N, K, cta, thread, nth):
    call, out, want = prepared(hooks, sizes, N, K)
    assert hooks.mxfp4_device_status(None) == 0
    hooks.mxfp4_test_stream_give_up(cta, thread, nth)
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


# Every call has the same tag here, as the replays of one graph do, and the workspace is left as the call before
# left it: a call must not take the arrivals of one that gave up for its own.
@pytest.mark.parametrize("sizes,N,K,cta,thread,nth", [c for c in CASES if c[0] != 1 or c[1] != 2112])
def test_a_replay_after_one_that_gave_up(hooks, sizes, N, K, cta, thread, nth):
    call, out, want = prepared(hooks, sizes, N, K)
    hooks.mxfp4_test_stream_tag(0x123456789ABCDE)
    try:
        for _ in range(3):
            hooks.mxfp4_test_stream_give_up(cta, thread, nth)
            assert call() == 0
            torch.cuda.synchronize()
            assert hooks.mxfp4_device_status(None) == TIMEOUT
            hooks.mxfp4_test_stream_give_up(-1, 0, 0)
            out.zero_()
            assert call() == 0
            torch.cuda.synchronize()
            assert hooks.mxfp4_device_status(None) == 0
            assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    finally:
        hooks.mxfp4_test_stream_tag(0)
