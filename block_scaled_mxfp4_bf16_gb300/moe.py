"""The mixture-of-experts and weight-only operators of the binding: mxfp4_gemv, mxfp4_grouped_gemm,
mxfp4_moe_route and mxfp4_moe_combine. As in the rest of the binding, the functions only check and
marshal arguments; every step runs in the library's CUDA kernels."""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import (Mxfp4Error, _check, _check_packed, _dev, _on, _stream, _workspace, load_library, mxfp4_prepack_b,
               mxfp4_prepack_b_size)

_NEED: dict = {}


def _need(query: str, device: torch.device, *sizes: int) -> int:
    """A workspace query, remembered per (device, sizes): it depends only on those."""
    key = (query, device.index, *sizes)
    need = _NEED.get(key)
    if need is None:
        need = getattr(load_library(), query)(*sizes)
        _NEED[key] = need
    return need


def _scratch(workspace, need: int, device: torch.device, stream, st: int) -> tuple:
    """(pointer, bytes) of the caller's workspace, or of the binding's own for this stream."""
    if workspace is None:
        workspace = _workspace(device, need, stream, st)
        if workspace is None:
            return None, 0
    else:
        _on(workspace, device, "workspace")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.nbytes


def _dense_rows(t: torch.Tensor) -> bool:
    """Whether the columns lie next to each other (strides of 0 or 1 element say nothing)."""
    return t.dim() == 2 and (t.stride(1) == 1 or t.shape[1] <= 1 or t.shape[0] == 0)


def _ld(t: torch.Tensor) -> int:
    """Row stride of a 2-D tensor; a single row has none that matters."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _bf16_rows(t: torch.Tensor, name: str) -> None:
    if t.dtype != torch.bfloat16 or not _dense_rows(t):
        raise ValueError(f"{name} must be a 2-D bf16 tensor with unit column stride")


def _empty(shape: tuple, dtype: torch.dtype, device: torch.device, stream) -> torch.Tensor:
    """An output of the call: its memory belongs to the stream that writes it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _out(t: torch.Tensor | None, shape: tuple, device: torch.device, name: str, stream) -> torch.Tensor:
    if t is None:
        return _empty(shape, torch.bfloat16, device, stream)
    _on(t, device, name)
    if t.dtype != torch.bfloat16 or tuple(t.shape) != shape or not _dense_rows(t):
        raise ValueError(f"{name} must be a bf16 {list(shape)} tensor with unit column stride")
    return t


def _index(t: torch.Tensor, shape: tuple, device: torch.device, name: str, dtype=torch.int32) -> None:
    if t.device != device or t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)} on {device}")


def mxfp4_gemv(x: torch.Tensor, packed_b: torch.Tensor, N: int, y: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y [M, N] bf16 = x . W^T for a few tokens, x [M, K] kept in bf16 (not quantized), W the MXFP4
    weights of `packed_b` (mxfp4_prepack_b): the weight-only product, on the weights mxfp4_gemm uses."""
    L = load_library()
    _dev(x, "x")
    _bf16_rows(x, "x")
    M, K = x.shape
    device = x.device
    if M and N:
        _check_packed(packed_b, N, K, device)
    y = _out(y, (M, N), device, "y", stream)
    st = _stream(stream)
    need = _need("mxfp4_gemv_workspace_size", device, M, N, K) if M and N else 0
    ws, ws_bytes = _scratch(workspace, need, device, stream, st)
    _check(L.mxfp4_gemv(x.data_ptr(), M, K, _ld(x), packed_b.data_ptr(), N, y.data_ptr(), _ld(y), ws, ws_bytes,
                        st), "mxfp4_gemv")
    return y


def mxfp4_prepack_experts(bq: torch.Tensor, bs: torch.Tensor, stream=None) -> torch.Tensor:
    """Pre-quantized weights of E experts (e2m1 [E, N, nblk*16], e8m0 [E, N, nblk]) -> uint8
    [E, mxfp4_prepack_b_size(N, K)], each row packed by mxfp4_prepack_b: the weights
    mxfp4_grouped_gemm reads."""
    if bq.dim() != 3 or bs.dim() != 3 or bq.shape[0] != bs.shape[0]:
        raise ValueError("bq [E, N, nblk*16] and bs [E, N, nblk] must be 3-D with the same E")
    _dev(bq, "bq")
    E, N, K = bq.shape[0], bq.shape[1], bq.shape[2] * 2
    size = mxfp4_prepack_b_size(N, K)
    if size == 0:
        raise Mxfp4Error(2, "mxfp4_prepack_b_size")
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
    L = load_library()
    _dev(a, "a")
    _bf16_rows(a, "a")
    tokens, K = a.shape
    if gated:
        if K % 2:
            raise ValueError("a gated product's a must have an even number of columns")
        K //= 2
    device = a.device
    if packed_b.dim() != 2 or not packed_b.is_contiguous():
        raise ValueError("packed_b must be a contiguous [E, bytes] buffer (mxfp4_prepack_experts)")
    E = packed_b.shape[0]
    if E and N:
        _check_packed(packed_b[0] if E > 1 else packed_b, N, K, device)
        if packed_b.shape[1] * packed_b.element_size() != mxfp4_prepack_b_size(N, K):
            raise ValueError(f"packed_b's rows must have mxfp4_prepack_b_size({N}, {K}) bytes")
    _index(offsets, (E + 1,), device, "offsets")
    if rows is None:
        R, rows_ptr = tokens, None
    else:
        R = rows.shape[0] if rows.dim() == 1 else -1
        _index(rows, (R,), device, "rows")
        rows_ptr = rows.data_ptr()
    c = _out(c, (R, N), device, "c", stream)
    st = _stream(stream)
    need = _need("mxfp4_grouped_gemm_workspace_size", device, R, E, N, K) if R and E and N else 0
    ws, ws_bytes = _scratch(workspace, need, device, stream, st)
    _check(L.mxfp4_grouped_gemm(a.data_ptr(), tokens, K, _ld(a), rows_ptr, offsets.data_ptr(), E,
                                packed_b.data_ptr(), N, c.data_ptr(), R, _ld(c), 1 if gated else 0, ws, ws_bytes, st),
           "mxfp4_grouped_gemm")
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
    L = load_library()
    _dev(logits, "logits")
    dtype = _LOGIT_TYPES.get(logits.dtype)
    if dtype is None or not _dense_rows(logits):
        raise ValueError("logits must be a 2-D fp32 or bf16 tensor with unit column stride")
    T, E = logits.shape
    if not 1 <= k <= min(E, 32):
        raise ValueError(f"k must lie in 1 .. min(E, 32) = {min(E, 32)}")
    device = logits.device
    weights = _empty((T, k), torch.float32, device, stream)
    experts = _empty((T, k), torch.int32, device, stream)
    offsets = _empty((E + 1,), torch.int32, device, stream)
    rows = _empty((T * k,), torch.int32, device, stream)
    slots = _empty((T, k), torch.int32, device, stream)
    st = _stream(stream)
    ws, ws_bytes = _scratch(workspace, _need("mxfp4_moe_route_workspace_size", device, T, E), device, stream, st)
    _check(L.mxfp4_moe_route(logits.data_ptr(), dtype, T, E, _ld(logits), k, 0 if renormalize else 1,
                             weights.data_ptr(), experts.data_ptr(), offsets.data_ptr(), rows.data_ptr(),
                             slots.data_ptr(), ws, ws_bytes, st), "mxfp4_moe_route")
    return MoeRouting(weights, experts, offsets, rows, slots)


def mxfp4_moe_combine(y: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor, out: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """out [T, N] bf16 = sum over j of weights[t, j] * y[slots[t, j]] (fp32 sums), y [R, N] bf16 in the
    grouped order; a slot outside [0, R) adds nothing."""
    L = load_library()
    _dev(y, "y")
    _bf16_rows(y, "y")
    R, N = y.shape
    if slots.dim() != 2:
        raise ValueError("slots must be [T, k]")
    T, k = slots.shape
    _index(slots, (T, k), y.device, "slots")
    _index(weights, (T, k), y.device, "weights", torch.float32)
    out = _out(out, (T, N), y.device, "out", stream)
    _check(L.mxfp4_moe_combine(y.data_ptr(), R, N, _ld(y), slots.data_ptr(), weights.data_ptr(), T, k,
                               out.data_ptr(), _ld(out), _stream(stream)), "mxfp4_moe_combine")
    return out
