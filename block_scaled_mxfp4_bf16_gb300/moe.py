"""The mixture-of-experts and weight-only operators of the binding: mxfp4_gemv, mxfp4_grouped_gemm,
mxfp4_moe_route and mxfp4_moe_combine. As in the rest of the binding, the functions only check and
marshal arguments; every step runs in the library's CUDA kernels.

These calls sit between short kernels in a decoding loop, where the host's time is the loop's time,
so each reads a tensor property once and leaves the reports of what is wrong to slower helpers."""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import (_PACKED_NEED, _WS, Mxfp4Error, _check, _check_packed, _current_capturing, _dev, _on, _raw_stream, _stream,
               _workspace, _writing, load_library, mxfp4_prepack_b, mxfp4_prepack_b_size)

_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_NEED: dict = {}
# without the check for a context, which a tensor on the device has already
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _need(query: str, device: int, *sizes: int) -> int:
    """A size query of the library for the current device, remembered: it depends on its arguments only."""
    key = (query, device, *sizes)
    need = _NEED.get(key)
    if need is None:
        need = getattr(load_library(), query)(*sizes)
        if need:
            _NEED[key] = need
    return need


def _begin(t: torch.Tensor, name: str, stream) -> tuple:
    """(stream, device) of a call whose first operand is `t`, which must live on the current CUDA device."""
    d = t.get_device()
    if d < 0 or d != _device():
        _dev(t, name)
    return _raw_stream(d) if stream is None and _raw_stream is not None else _stream(stream), d


def _scratch(workspace, need: int, t: torch.Tensor, stream, st: int, device: int) -> tuple:
    """(pointer, bytes) of the caller's workspace or of this thread's default one for the stream, and the
    tensor, which has to live until the call is enqueued."""
    if workspace is not None:
        _on(workspace, t.device, "workspace")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    elif need == 0:
        return None, 0, None
    else:
        if stream is None and not _current_capturing():
            workspace = _WS.held.get((device, st))
        if workspace is None or workspace.nbytes < need:
            workspace = _workspace(t.device, need, stream, st)
    return workspace.data_ptr(), workspace.nbytes, workspace


def _rows_of(t: torch.Tensor, name: str) -> int:
    """The row stride of a 2-D tensor whose columns lie next to each other (a single row has none
    that matters)."""
    if t.dim() == 2:
        rows, cols = t.shape
        ld, step = t.stride()
        if step == 1 or cols <= 1 or rows == 0:
            return ld if rows > 1 else cols
    raise ValueError(f"{name} must be a 2-D tensor with unit column stride")


def _bf16_rows(t: torch.Tensor, name: str) -> int:
    if t.dtype != _BF16:
        raise ValueError(f"{name} must be a bf16 tensor")
    return _rows_of(t, name)


# the allocation that compiled graphs use: 0.6 us a tensor less than torch.empty
_empty_strided = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None), "_empty_strided_cuda", None)


def _empty(shape: tuple, dtype: torch.dtype, t: torch.Tensor, stream) -> torch.Tensor:
    """An output of a call, on t's (the current) device: its memory belongs to the stream that writes it."""
    if stream is None:
        if _empty_strided is not None:
            return _empty_strided(shape, (shape[1], 1) if len(shape) == 2 else (1,), dtype)
        return torch.empty(shape, dtype=dtype, device=t.device)
    with _writing(stream, t.device):
        return torch.empty(shape, dtype=dtype, device=t.device)


def _out(out: torch.Tensor | None, shape: tuple, t: torch.Tensor, name: str, stream) -> tuple:
    """(output, its row stride): the caller's, checked, or a new one."""
    if out is None:
        return _empty(shape, _BF16, t, stream), shape[1]
    _on(out, t.device, name)
    if tuple(out.shape) != shape:
        raise ValueError(f"{name} must be a {list(shape)} tensor")
    return out, _bf16_rows(out, name)


def _index(t: torch.Tensor, shape: tuple, like: torch.Tensor, name: str, dtype=_I32) -> int:
    """Pointer of a dense index (or weight) tensor on the operands' device."""
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != like.get_device():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)} on {like.device}")
    return t.data_ptr()


def mxfp4_gemv(x: torch.Tensor, packed_b: torch.Tensor, N: int, y: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y [M, N] bf16 = x . W^T for a few tokens, x [M, K] bf16 and not quantized (an element is held to within
    2^-22 of its 1x32 block's largest magnitude), W the MXFP4 weights of `packed_b` (mxfp4_prepack_b): the
    weight-only product, on the weights mxfp4_gemm uses."""
    st, device = _begin(x, "x", stream)
    ldx = _bf16_rows(x, "x")
    M, K = x.shape
    need = 0
    if M and N:
        _check_packed(packed_b, N, K, x.device)
        need = _need("mxfp4_gemv_workspace_size", device, M, N, K)
    y, ldy = _out(y, (M, N), x, "y", stream)
    ws, ws_bytes, _held = _scratch(workspace, need, x, stream, st, device)
    status = load_library().mxfp4_gemv(x.data_ptr(), M, K, ldx, packed_b.data_ptr(), N, y.data_ptr(), ldy, ws, ws_bytes,
                                       st)
    if status:
        _check(status, "mxfp4_gemv")
    return y


def mxfp4_prepack_experts(bq: torch.Tensor, bs: torch.Tensor, stream=None) -> torch.Tensor:
    """Pre-quantized weights of E experts (e2m1 [E, N, nblk*16], e8m0 [E, N, nblk]) -> uint8
    [E, mxfp4_prepack_b_size(N, K)], each row packed by mxfp4_prepack_b: the weights
    mxfp4_grouped_gemm reads. Their memory belongs to the stream that writes them."""
    if bq.dim() != 3 or bs.dim() != 3 or bq.shape[0] != bs.shape[0]:
        raise ValueError("bq [E, N, nblk*16] and bs [E, N, nblk] must be 3-D with the same E")
    _dev(bq, "bq")
    E, N, K = bq.shape[0], bq.shape[1], bq.shape[2] * 2
    size = mxfp4_prepack_b_size(N, K)
    if size == 0:
        raise Mxfp4Error(2, "mxfp4_prepack_b_size")
    with _writing(stream, bq.device):
        store = torch.empty(E * size + 1024, dtype=torch.uint8, device=bq.device)
    off = (-store.data_ptr()) % 1024
    packed = store[off:off + E * size].view(E, size)
    for e in range(E):
        mxfp4_prepack_b(bq[e], bs[e], packed=packed[e], stream=stream)
    return packed


def mxfp4_grouped_gemm(a: torch.Tensor, packed_b: torch.Tensor, offsets: torch.Tensor, N: int,
                       rows: torch.Tensor | None = None, gated: bool = False, c: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """C [R, N] bf16, rows sorted by expert: C[r] = MXFP4(a[rows[r]]) . MXFP4(W_e)^T for the rows
    offsets[e] <= r < offsets[e+1] of expert e. `packed_b`: mxfp4_prepack_experts' weights; `offsets`
    [E+1] and `rows` [R]: int32 on the device, as mxfp4_moe_route returns them (rows None: row r of
    `a`). gated: a's rows are [g, u] and silu(g) * u is the product's input, K = a.shape[1] / 2.
    Rows of C that belong to no expert are not written."""
    st, device = _begin(a, "a", stream)
    lda = _bf16_rows(a, "a")
    tokens, K = a.shape
    if gated:
        if K % 2:
            raise ValueError("a gated product's a must have an even number of columns")
        K //= 2
    if packed_b.dim() != 2 or not packed_b.is_contiguous():
        raise ValueError("packed_b must be a contiguous [E, bytes] buffer (mxfp4_prepack_experts)")
    E = packed_b.shape[0]
    if E and N:
        _check_packed(packed_b, N, K, a.device)
        if packed_b.nbytes != E * _PACKED_NEED[(N, K)]:
            raise ValueError(f"packed_b's rows must have mxfp4_prepack_b_size({N}, {K}) bytes")
    offsets_ptr = _index(offsets, (E + 1,), a, "offsets")
    if rows is None:
        R, rows_ptr = tokens, None
    else:
        R = rows.shape[0] if rows.dim() == 1 else -1
        rows_ptr = _index(rows, (R,), a, "rows")
    c, ldc = _out(c, (R, N), a, "c", stream)
    need = _need("mxfp4_grouped_gemm_workspace_size", device, R, E, N, K) if R and E and N else 0
    ws, ws_bytes, _held = _scratch(workspace, need, a, stream, st, device)
    status = load_library().mxfp4_grouped_gemm(a.data_ptr(), tokens, K, lda, rows_ptr, offsets_ptr, E,
                                               packed_b.data_ptr(), N, c.data_ptr(), R, ldc, 1 if gated else 0, ws,
                                               ws_bytes, st)
    if status:
        _check(status, "mxfp4_grouped_gemm")
    return c


class MoeRouting(NamedTuple):
    """What mxfp4_moe_route returns: weights fp32 [T, k] and experts int32 [T, k] per token, and the
    grouping by expert: offsets int32 [E+1], rows int32 [T*k] (the token of each sorted row), slots
    int32 [T, k] (the sorted row of each pair). -1 where nothing is routed."""
    weights: torch.Tensor
    experts: torch.Tensor
    offsets: torch.Tensor
    rows: torch.Tensor
    slots: torch.Tensor


_LOGIT_TYPES = {torch.float32: 0, torch.bfloat16: 1}


def mxfp4_moe_route(logits: torch.Tensor, k: int, renormalize: bool = True, workspace: torch.Tensor | None = None,
                    stream=None) -> MoeRouting:
    """Top-k routing of logits [T, E] (fp32 or bf16): the k largest per token (ties to the lower index;
    -inf and NaN are masks), their softmax weights (over the k, or with renormalize=False over all
    experts), and the token-expert pairs grouped by expert."""
    st, device = _begin(logits, "logits", stream)
    dtype = _LOGIT_TYPES.get(logits.dtype)
    if dtype is None:
        raise ValueError("logits must be an fp32 or bf16 tensor")
    ld = _rows_of(logits, "logits")
    T, E = logits.shape
    if not 1 <= k <= min(E, 32):
        raise ValueError(f"k must lie in 1 .. min(E, 32) = {min(E, 32)}")
    if stream is None and _empty_strided is not None:
        weights = _empty_strided((T, k), (k, 1), _F32)
        experts = _empty_strided((T, k), (k, 1), _I32)
        offsets = _empty_strided((E + 1,), (1,), _I32)
        rows = _empty_strided((T * k,), (1,), _I32)
        slots = _empty_strided((T, k), (k, 1), _I32)
    else:
        weights, experts, offsets, rows, slots = (
            _empty(shape, dtype, logits, stream)
            for shape, dtype in (((T, k), _F32), ((T, k), _I32), ((E + 1,), _I32), ((T * k,), _I32), ((T, k), _I32)))
    ws, ws_bytes, _held = _scratch(workspace, _need("mxfp4_moe_route_workspace_size", device, T, E), logits, stream, st, device)
    status = load_library().mxfp4_moe_route(logits.data_ptr(), dtype, T, E, ld, k, 0 if renormalize else 1,
                                            weights.data_ptr(), experts.data_ptr(), offsets.data_ptr(),
                                            rows.data_ptr(), slots.data_ptr(), ws, ws_bytes, st)
    if status:
        _check(status, "mxfp4_moe_route")
    return MoeRouting(weights, experts, offsets, rows, slots)


def mxfp4_moe_combine(y: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor, out: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """out [T, N] bf16 = sum over j of weights[t, j] * y[slots[t, j]] (fp32 sums), y [R, N] bf16 in the
    grouped order; a slot outside [0, R) adds nothing."""
    st, _ = _begin(y, "y", stream)
    ldy = _bf16_rows(y, "y")
    R, N = y.shape
    if slots.dim() != 2:
        raise ValueError("slots must be [T, k]")
    T, k = slots.shape
    slots_ptr = _index(slots, (T, k), y, "slots")
    weights_ptr = _index(weights, (T, k), y, "weights", _F32)
    out, ldo = _out(out, (T, N), y, "out", stream)
    status = load_library().mxfp4_moe_combine(y.data_ptr(), R, N, ldy, slots_ptr, weights_ptr, T, k, out.data_ptr(), ldo,
                                              st)
    if status:
        _check(status, "mxfp4_moe_combine")
    return out
