"""Calls that pass no workspace, on the GPU: several host threads on one stream must get the results that one
thread gets, whatever order their calls' kernels are enqueued in, and a graph captured from such calls must
keep to memory of its own."""
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


def layer(seed, tokens):
    """A mixture-of-experts pass and a weight-only product, no workspace passed: (call, larger call)."""
    import block_scaled_mxfp4_bf16_gb300 as mx
    E, k, hidden, inner = 4, 2, 1024, 256
    w13, _ = weights(E, 2 * inner, hidden, seed=seed)
    w2, _ = weights(E, hidden, inner, seed=seed + 1)

    def of(T):
        x = workloads.random_bf16(T, hidden, seed=seed + T).cuda()
        logits = torch.randn(T, E, generator=torch.Generator().manual_seed(seed + T)).cuda()

        def call():
            r = mx.mxfp4_moe_route(logits, k)
            h = mx.mxfp4_grouped_gemm(x, w13, r.offsets, 2 * inner, rows=r.rows)
            y = mx.mxfp4_grouped_gemm(h, w2, r.offsets, hidden, gated=True)
            return [mx.mxfp4_moe_combine(y, r.slots, r.weights), mx.mxfp4_gemv(x[:5], w13[0], 2 * inner),
                    mx.mxfp4_gemm(x, w13[1], 2 * inner, path=2)]
        return call
    return of(tokens), of(20 * tokens)


def test_a_larger_call_after_the_capture_leaves_the_graph_its_memory():
    import block_scaled_mxfp4_bf16_gb300 as mx
    call, larger = layer(7, 300)
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        want = [o.clone() for o in call()]          # warm-up: the stream's default workspace is there
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            outs = call()
        larger()                                    # replaces the default workspace by a larger one
        torch.cuda.synchronize()
        others = [torch.full((n << 20,), 0x5A, dtype=torch.uint8, device="cuda") for n in (1, 1, 2, 4, 8, 16, 32)]
        for _ in range(3):
            for o in outs:
                o.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert equal(outs, want)
    assert all(bool((o == 0x5A).all()) for o in others), "a replay wrote into another tensor's memory"
    assert mx.mxfp4_device_status() == 0


def test_graphs_of_one_capture_stream_replay_side_by_side():
    import block_scaled_mxfp4_bf16_gb300 as mx
    calls = [layer(20 + i, 300)[0] for i in range(2)]
    wants = [[o.clone() for o in call()] for call in calls]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for call in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):               # the default capture stream, the same for both
            outs.append(call())
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, wants):
        assert equal(o, w)
    assert mx.mxfp4_device_status() == 0


def test_packed_experts_take_no_memory_the_current_stream_may_still_read():
    import block_scaled_mxfp4_bf16_gb300 as mx
    E, N, K = 3, 256, 512
    bq, bs = mx.mxfp4_quantize(workloads.random_bf16(E * N, K, seed=1).cuda())
    bq, bs = bq.view(E, N, -1), bs.view(E, N, -1)
    want = mx.mxfp4_prepack_experts(bq, bs)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    read = torch.arange(want.nbytes + 1024, device="cuda").to(torch.uint8)
    keep = read.clone()
    torch.cuda._sleep(20_000_000)            # about 10 ms: the copy is still queued when its source is dropped
    copy = read.clone()
    del read
    got = mx.mxfp4_prepack_experts(bq, bs, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(copy, keep)
