"""Calls that pass no workspace, on the GPU: several host threads on one stream must get the results that one
thread gets, whatever order their calls' kernels are enqueued in."""
import threading

import pytest
import torch

from block_scaled_mxfp4_bf16_gb300 import workloads
from moe_testlib import weights

pytestmark = pytest.mark.gpu


def equal(a, b):
    return all(torch.equal(x.view(torch.int16) if x.dtype == torch.bfloat16 else x,
                           y.view(torch.int16) if y.dtype == torch.bfloat16 else y) for x, y in zip(a, b))


def two_launch_calls(seed):
    """Calls of two kernels that hand something over in the workspace, each with inputs of its own: a
    function that makes the call and returns its outputs."""
    import block_scaled_mxfp4_bf16_gb300 as mx
    E, N, K = 4, 256, 1024
    packed, _ = weights(E, N, K, seed=seed)
    sizes = [90, 0, 130, 200]
    offsets = torch.tensor([0, 90, 90, 220, 420], dtype=torch.int32, device="cuda")
    a = workloads.random_bf16(sum(sizes), K, seed=seed + 1).cuda()
    x = workloads.random_bf16(5, K, seed=seed + 2).cuda()
    logits = torch.randn(6000, 33, generator=torch.Generator().manual_seed(seed)).cuda()
    return [lambda: [mx.mxfp4_grouped_gemm(a, packed, offsets, N)], lambda: [mx.mxfp4_gemv(x, packed[0], N)],
            lambda: list(mx.mxfp4_moe_route(logits, 8)), lambda: [mx.mxfp4_gemm(a, packed[1], N, path=2)]]


def test_threads_on_one_stream():
    import block_scaled_mxfp4_bf16_gb300 as mx
    sets = [two_launch_calls(100 * t) for t in range(4)]
    want = [[call() for call in calls] for calls in sets]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    got, errors = {}, []
    start = threading.Barrier(len(sets))

    def worker(t):
        try:
            with torch.cuda.stream(stream):
                start.wait()
                got[t] = [[call() for call in sets[t]] for _ in range(60)]
        except Exception as e:   # reported below, on the main thread
            errors.append((t, repr(e)))

    threads = [threading.Thread(target=worker, args=(t,)) for t in range(len(sets))]
    for th in threads:
        th.start()
    for th in threads:
        th.join(timeout=120)
    torch.cuda.synchronize()
    assert not errors, errors
    assert mx.mxfp4_device_status() == 0
    for t, runs in got.items():
        for outs in runs:
            for i, (o, w) in enumerate(zip(outs, want[t])):
                assert equal(o, w), (t, i)
    assert len(got) == len(sets)
