"""The binding's default workspaces, on the CPU: which calls share one. Calls that do must be ordered;
two threads' calls on one stream are not, since a call of several kernels enqueues them with the
interpreter's lock released between them."""
import contextlib
import threading
import types

import pytest
import torch

import block_scaled_mxfp4_bf16_gb300 as mx
from block_scaled_mxfp4_bf16_gb300 import moe
from test_binding_checks import dev
from test_moe_checks import _MoeLib, bf16, i32, packed

CPU = torch.device("cpu")


@pytest.fixture
def made(monkeypatch):
    """Workspaces on the CPU: every one made, in order."""
    fake = _MoeLib(mx.load_library())
    tensors = []
    real_empty = torch.empty

    def empty(*shape, **kw):
        t = real_empty(*shape, **kw)
        if kw.get("dtype") is torch.uint8 and len(shape) == 1:
            tensors.append(t)
            world.owners.append(world.stream)
        return t
    monkeypatch.setattr(mx, "load_library", lambda: fake)
    monkeypatch.setattr(moe, "load_library", lambda: fake)
    monkeypatch.setattr(moe, "_NEED", {})
    monkeypatch.setattr(mx, "_WS", type(mx._WS)())
    monkeypatch.setattr(moe, "_WS", mx._WS)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)   # a CPU tensor's get_device()
    world = types.SimpleNamespace(tensors=tensors, lib=fake, stream=0, capturing=False, owners=[])   # stream: current
    for module in (mx, moe):
        monkeypatch.setattr(module, "_raw_stream", lambda device: world.stream)
        monkeypatch.setattr(module, "_current_capturing", lambda: world.capturing, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=world.stream))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda st, device=None: st)

    @contextlib.contextmanager
    def on(stream):
        before, world.stream = world.stream, stream
        yield
        world.stream = before
    monkeypatch.setattr(torch.cuda, "stream", on)
    return world


def in_thread(f):
    out = []
    t = threading.Thread(target=lambda: out.append(f()))
    t.start()
    t.join()
    return out[0]


def test_a_thread_keeps_its_workspace_from_call_to_call(made):
    first = mx._workspace(CPU, 5000, 0, 0)
    assert first.numel() >= 5000 and mx._workspace(CPU, 5000, 0, 0) is first
    assert mx._workspace(CPU, 4000, 0, 0) is first, "a smaller call takes the one there is"
    made.stream = 1
    assert mx._workspace(CPU, 5000, 1, 1) is not first, "another stream's calls are not ordered with it"
    made.stream = 0
    grown = mx._workspace(CPU, 3 << 20, 0, 0)
    assert grown.numel() >= 3 << 20 and mx._workspace(CPU, 5000, 0, 0) is grown
    assert mx._workspace(CPU, 0, 0, 0) is None


def test_two_threads_on_one_stream_have_a_workspace_each(made):
    here = mx._workspace(CPU, 5000, 0, 0)
    there = in_thread(lambda: mx._workspace(CPU, 5000, 0, 0))
    assert there.data_ptr() != here.data_ptr()


def _workspace_argument(made, call):
    call()
    name, args = made.lib.calls[-1]
    return args[{"mxfp4_gemv": 8, "mxfp4_grouped_gemm": 13}[name]]


@pytest.mark.parametrize("op", ["gemv", "grouped"])
def test_two_threads_calls_hand_over_different_workspaces(made, op):
    if op == "gemv":
        def call():
            mx.mxfp4_gemv(bf16(3, 256), packed(1, 128, 256)[0], 128, y=bf16(3, 128), stream=0)
    else:
        def call():
            mx.mxfp4_grouped_gemm(bf16(6, 256), packed(3, 128, 256), i32(0, 2, 4, 6), 128, c=bf16(6, 128), stream=0)
    here = _workspace_argument(made, call)
    assert here == _workspace_argument(made, call)
    assert in_thread(lambda: _workspace_argument(made, call)) != here


def test_prepared_calls_have_a_workspace_of_their_own(made, monkeypatch):
    # any thread may run them, beside the calls of the thread that prepared them
    monkeypatch.setattr(mx, "_ws_need", lambda *a: 5000)
    a, b, c = bf16(8, 512), packed(1, 256, 512)[0], bf16(8, 256)
    seen = {mx._workspace(CPU, 5000, 0, 0).data_ptr()}
    calls = [mx.prepare_gemm(a, b, 256, c, stream=0) for _ in range(2)]
    for name, args in made.lib.calls:
        if name == "mxfp4_call_create":
            seen.add(args[8])
    assert len(seen) == 3
    del calls


@pytest.mark.parametrize("op", ["gemv", "grouped"])
def test_a_captured_call_has_a_workspace_of_its_own(made, op):
    # a graph keeps the address: it must be neither the default one, which a larger call replaces, nor
    # one that is kept for the calls after the capture
    if op == "gemv":
        def call():
            mx.mxfp4_gemv(bf16(3, 256), packed(1, 128, 256)[0], 128, y=bf16(3, 128))
    else:
        def call():
            mx.mxfp4_grouped_gemm(bf16(6, 256), packed(3, 128, 256), i32(0, 2, 4, 6), 128, c=bf16(6, 128))
    eager = _workspace_argument(made, call)
    held = dict(mx._WS.held)
    made.capturing = True
    kept = len(made.tensors)
    first = _workspace_argument(made, call)
    assert len(made.tensors) == kept + 1 and first == made.tensors[-1].data_ptr() != eager
    assert mx._WS.held == held, "memory of the graph's pool is kept for calls outside it"
    made.capturing = False
    assert _workspace_argument(made, call) == eager


def test_the_captured_gemm_has_a_workspace_of_its_own(made, monkeypatch):
    monkeypatch.setattr(mx, "_ws_need", lambda *a: 5000)
    a, b, c = bf16(8, 512), packed(1, 256, 512)[0], bf16(8, 256)

    def pointer():
        mx.mxfp4_gemm(a, b, 256, c=c)
        return made.lib.calls[-1][1][8]
    eager = pointer()
    made.capturing = True
    assert pointer() != eager
    made.capturing = False
    assert pointer() == eager


def test_memory_belongs_to_the_stream_that_writes_it(made):
    # what the current stream freed may still be read by work queued there
    mx._workspace(CPU, 5000, 7, 7)
    mx._workspace(CPU, 5000, None, 0)
    assert made.owners == [7, 0]
    bq, bs = (dev(torch.zeros(3, 128, n, dtype=torch.uint8)) for n in (128, 8))
    mx.mxfp4_prepack_experts(bq, bs, stream=9)
    mx.mxfp4_prepack_experts(bq, bs)
    assert made.owners == [7, 0, 9, 0] and made.stream == 0
