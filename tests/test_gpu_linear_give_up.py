"""Products with an epilogue in which one thread's bounded wait counts as run out: the kernel ends all the same, the
status says so, and the next call on the same workspace gives the right result (see test_gpu_give_up)."""
import ctypes

import pytest
import torch

from block_scaled_mxfp4_bf16_gb300 import workloads
from test_gpu_gated_linear import gated_weights
from moe_testlib import weights
from test_gpu_give_up import TIMEOUT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hooks():
    from block_scaled_mxfp4_bf16_gb300 import build
    L = ctypes.CDLL(build.build_variant("hooks", ["-DMXFP4_TEST_HOOKS"]))
    vp, i64, sz, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
    L.mxfp4_test_stream_give_up.argtypes = [i32, i32, i32]
    L.mxfp4_test_stream_give_up.restype = None
    L.mxfp4_linear.argtypes = [vp, i64, i64, i64, vp, i64, vp, i32, i32, vp, i64, vp, i64, vp, sz, vp]
    L.mxfp4_gated_linear.argtypes = [vp, i64, i64, i64, vp, i64, vp, i32, i32, vp, i64, vp, sz, vp]
    L.mxfp4_device_status.argtypes = [vp]
    for name in ("mxfp4_linear_workspace_size", "mxfp4_gated_linear_workspace_size"):
        getattr(L, name).restype = sz
        getattr(L, name).argtypes = [i64] * 3
    yield L
    L.mxfp4_test_stream_give_up(-1, 0, 0)


# operator, M, columns, K, then the thread: CTA, thread, nth wait of its warp: epilogue warps (128 .. 383) in whole units, with
# and without tensor copies, and in split ones; warps that write scale factors (384 .. 639 of a pair)
CASES = [
    ("linear", 1500, 4104, 7168, 5, 140, 0), ("linear", 1500, 4104, 7168, 6, 300, 1), ("linear", 1500, 4101, 7168, 5, 200, 0),
    ("linear", 8192, 4096, 7168, 3, 130, 8), ("linear", 8192, 4096, 7168, 8, 383, 7), ("linear", 1000, 7168, 2048, 4, 160, 1),
    ("linear", 1500, 4104, 7168, 2, 400, 6), ("gated", 1500, 2056, 7168, 5, 140, 0), ("gated", 4096, 3500, 4096, 9, 250, 3),
]


@pytest.mark.parametrize("op,M,columns,K,cta,thread,nth", CASES)
def test_a_wait_that_runs_out_ends_the_kernel(hooks, op, M, columns, K, cta, thread, nth):
    import block_scaled_mxfp4_bf16_gb300 as mx
    st = torch.cuda.current_stream().cuda_stream
    x = workloads.random_bf16(M, K, seed=4).cuda()
    if op == "linear":
        packed = weights(1, columns, K, seed=3)[0][0]
        r = workloads.random_bf16(M, columns, seed=5).cuda()
        want = mx.mxfp4_linear(x, packed, columns, activation="silu", residual=r)
        ws = torch.full((max(1, hooks.mxfp4_linear_workspace_size(M, columns, K)),), 0xEE, dtype=torch.uint8, device="cuda")
    else:
        packed = gated_weights(1, columns, K, seed=3)[0][0]
        want = mx.mxfp4_gated_linear(x, packed, columns)
        ws = torch.full((max(1, hooks.mxfp4_gated_linear_workspace_size(M, columns, K)),), 0xEE, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(want)

    def call():
        if op == "linear":
            return hooks.mxfp4_linear(x.data_ptr(), M, K, K, packed.data_ptr(), columns, None, 0, 2, r.data_ptr(), columns,
                                      out.data_ptr(), columns, ws.data_ptr(), ws.nbytes, st)
        return hooks.mxfp4_gated_linear(x.data_ptr(), M, K, K, packed.data_ptr(), columns, None, 0, 2, out.data_ptr(), columns,
                                        ws.data_ptr(), ws.nbytes, st)
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
