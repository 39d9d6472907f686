"""The products with an epilogue: mxfp4_linear (bias, activation, residual), mxfp4_gated_linear (two projections,
the activation and the product of a gated feed-forward block) and its form for experts' groups of rows. As in the
rest of the binding, the functions only check and marshal arguments; every step runs in the library's CUDA kernels.

A call of a few tokens takes the GPU 2 to 5 us and the host 7 or more, half as much again on a busy one: it reads every tensor property once, keeps the
sizes that the library answers by shape, and leaves the reports of what is wrong to slower helpers."""
from __future__ import annotations

import torch

from . import (Mxfp4Error, _check, _dev, _on, _raw_stream, _remember, _stream, _writing, load_library,
               mxfp4_prepack_b_size)
from .moe import _BF16, _F32, _bf16_rows, _device, _empty_strided, _index, _out, _scratch

# the C ABI's activations
ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
_BIAS_TYPES = {_F32: 0, _BF16: 1}


def _activation(name) -> int:
    """For a name that ACTIVATIONS does not have."""
    raise ValueError(f"activation must be one of {', '.join(str(n) for n in ACTIVATIONS)}, not {name!r}")


def _bias(bias: torch.Tensor, shape: tuple, like: torch.Tensor) -> tuple:
    """(pointer, C type) of a dense fp32 or bf16 bias."""
    dtype = _BIAS_TYPES.get(bias.dtype)
    if dtype is None:
        raise ValueError("bias must be an fp32 or bf16 tensor")
    return _index(bias, shape, like, "bias", bias.dtype), dtype


# (bytes of one group's packed weights, bytes of workspace) by function, device and sizes; both depend on these only
_SIZES: dict = {}


def _sizes(key: tuple) -> tuple:
    query, packed_size, device, *sizes = key
    known = (packed_size(*sizes[-2:]), getattr(load_library(), query)(*sizes))  # the current device is theirs
    if known[0]:
        _remember(_SIZES, key, known)
    return known


def _too_small(name: str, what: str, need: int) -> None:
    raise ValueError(f"{name} must be a contiguous CUDA buffer of at least {what} = {need} bytes on the device of the"
                     " other operands")


def _rows_and_stride(t: torch.Tensor, name: str) -> tuple:
    """(rows, columns, row stride) of a bf16 matrix whose columns lie next to each other."""
    if t.dtype is _BF16 and t.is_contiguous():
        shape = t.shape
        if len(shape) == 2:
            return *shape, shape[1]
    ld = _bf16_rows(t, name)
    return *t.shape, ld


def mxfp4_linear(x: torch.Tensor, packed_b: torch.Tensor, N: int, bias: torch.Tensor | None = None,
                 activation: str | None = None, residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out [M, N] bf16 = act(MXFP4(x) . MXFP4(B)^T + bias) + residual, rounded once: mxfp4_gemm with what follows it.
    `packed_b`: mxfp4_prepack_b's; `bias` [N] fp32 or bf16; `activation`: none, relu, silu, gelu (by the normal
    distribution function) or gelu_tanh; `residual` [M, N] bf16 with any row stride of N or more, which `out` may be
    itself (but not where the residual is x)."""
    device = x.get_device()
    if device < 0 or device != _device():
        _dev(x, "x")
    st = _raw_stream(device) if stream is None and _raw_stream is not None else _stream(stream)
    M, K, ldx = _rows_and_stride(x, "x")
    act = ACTIVATIONS.get(activation)
    if act is None:
        _activation(activation)
    need = 0
    if M and N:
        key = ("mxfp4_linear_workspace_size", mxfp4_prepack_b_size, device, M, N, K)
        known = _SIZES.get(key) or _sizes(key)
        need = known[1]
        if not known[0] or packed_b.nbytes < known[0] or not packed_b.is_contiguous() or packed_b.get_device() != device:
            _too_small("packed_b", f"mxfp4_prepack_b_size({N}, {K})", known[0])
    bias_ptr, bias_type = (None, 0) if bias is None else _bias(bias, (N,), x)
    res_ptr, ldr = None, 0
    if residual is not None:
        if residual.get_device() != device:
            _on(residual, x.device, "residual")
        rows, cols, ldr = _rows_and_stride(residual, "residual")
        if rows != M or cols != N:
            raise ValueError(f"residual must be a [{M}, {N}] tensor")
        res_ptr = residual.data_ptr()
    if out is None and stream is None and _empty_strided is not None:
        out, ldo = _empty_strided((M, N), (N, 1), _BF16), N
    else:
        out, ldo = _out(out, (M, N), x, "out", stream)
    if need or workspace is not None:
        ws, ws_bytes, _held = _scratch(workspace, need, x, stream, st, device)
    else:
        ws, ws_bytes = None, 0
    status = load_library().mxfp4_linear(x.data_ptr(), M, K, ldx, packed_b.data_ptr(), N, bias_ptr, bias_type, act,
                                         res_ptr, ldr, out.data_ptr(), ldo, ws, ws_bytes, st)
    if status:
        _check(status, "mxfp4_linear")
    return out


def mxfp4_prepack_gated_size(I: int, K: int) -> int:
    return int(load_library().mxfp4_prepack_gated_size(I, K))


def _quantized_shape(bq: torch.Tensor, bs: torch.Tensor, dims: int) -> tuple:
    """(rows, K) of quantized gate and up weights, checked."""
    _dev(bq, "bq")
    _on(bs, bq.device, "bs")
    if bq.dim() != dims or bs.dim() != dims or not bq.is_contiguous() or not bs.is_contiguous():
        raise ValueError("bq and bs must be contiguous and have the same number of dimensions")
    if bq.element_size() != 1 or bs.element_size() != 1:
        raise ValueError("bq and bs must be byte tensors")
    K = bq.shape[-1] * 2
    if tuple(bs.shape) != (*bq.shape[:-1], K // 32) or bq.shape[-2] % 2:
        raise ValueError("bq [.., 2I, nblk*16] and bs [.., 2I, nblk] must be consistent, with an even number of rows")
    return bq.shape[-2] // 2, K


def _gated_bytes(I: int, K: int) -> int:
    size = mxfp4_prepack_gated_size(I, K)
    if size == 0:
        raise Mxfp4Error(2, "mxfp4_prepack_gated_size")
    return size


def mxfp4_prepack_gated(bq: torch.Tensor, bs: torch.Tensor, packed: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """Pre-quantized gate and up projections (e2m1 [2I, nblk*16], e8m0 [2I, nblk], the gate's I rows first) -> the
    packed weights of mxfp4_gated_linear. New memory belongs to the stream that writes it."""
    I, K = _quantized_shape(bq, bs, 2)
    size = _gated_bytes(I, K)
    if packed is None:
        with _writing(stream, bq.device):
            packed = torch.empty(size + 1024, dtype=torch.uint8, device=bq.device)
        off = (-packed.data_ptr()) % 1024
        packed = packed[off:off + size]
    elif packed.device != bq.device or packed.nbytes < size or not packed.is_contiguous():
        raise ValueError(f"packed must be a contiguous buffer of at least {size} bytes on {bq.device}")
    _check(load_library().mxfp4_prepack_gated(bq.data_ptr(), bs.data_ptr(), I, K, packed.data_ptr(), _stream(stream)),
           "mxfp4_prepack_gated")
    return packed


def mxfp4_prepack_gated_experts(bq: torch.Tensor, bs: torch.Tensor, stream=None) -> torch.Tensor:
    """Pre-quantized gate and up projections of E experts (e2m1 [E, 2I, nblk*16], e8m0 [E, 2I, nblk]) -> uint8
    [E, mxfp4_prepack_gated_size(I, K)], the weights mxfp4_grouped_gated_linear reads. Their memory belongs to the
    stream that writes them."""
    I, K = _quantized_shape(bq, bs, 3)
    E, size = bq.shape[0], _gated_bytes(I, K)
    with _writing(stream, bq.device):
        store = torch.empty(E * size + 1024, dtype=torch.uint8, device=bq.device)
    off = (-store.data_ptr()) % 1024
    packed = store[off:off + E * size].view(E, size)
    for e in range(E):
        mxfp4_prepack_gated(bq[e], bs[e], packed=packed[e], stream=stream)
    return packed


def mxfp4_gated_linear(x: torch.Tensor, packed_gu: torch.Tensor, I: int, bias: torch.Tensor | None = None,
                       activation: str | None = "silu", out: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out [M, I] bf16 = act(MXFP4(x) . Wg^T + bias[:I]) * (MXFP4(x) . Wu^T + bias[I:]), rounded once: the first half
    of a gated feed-forward block in one product. `packed_gu`: mxfp4_prepack_gated's; `bias` [2I] fp32 or bf16;
    `activation` as for mxfp4_linear."""
    device = x.get_device()
    if device < 0 or device != _device():
        _dev(x, "x")
    st = _raw_stream(device) if stream is None and _raw_stream is not None else _stream(stream)
    M, K, ldx = _rows_and_stride(x, "x")
    act = ACTIVATIONS.get(activation)
    if act is None:
        _activation(activation)
    need = 0
    if M and I:
        key = ("mxfp4_gated_linear_workspace_size", mxfp4_prepack_gated_size, device, M, I, K)
        known = _SIZES.get(key) or _sizes(key)
        need = known[1]
        if not known[0] or packed_gu.nbytes < known[0] or not packed_gu.is_contiguous() or packed_gu.get_device() != device:
            _too_small("packed_gu", f"mxfp4_prepack_gated_size({I}, {K})", known[0])
    bias_ptr, bias_type = (None, 0) if bias is None else _bias(bias, (2 * I,), x)
    if out is None and stream is None and _empty_strided is not None:
        out, ldo = _empty_strided((M, I), (I, 1), _BF16), I
    else:
        out, ldo = _out(out, (M, I), x, "out", stream)
    if need or workspace is not None:
        ws, ws_bytes, _held = _scratch(workspace, need, x, stream, st, device)
    else:
        ws, ws_bytes = None, 0
    status = load_library().mxfp4_gated_linear(x.data_ptr(), M, K, ldx, packed_gu.data_ptr(), I, bias_ptr, bias_type,
                                               act, out.data_ptr(), ldo, ws, ws_bytes, st)
    if status:
        _check(status, "mxfp4_gated_linear")
    return out


def mxfp4_grouped_gated_linear(a: torch.Tensor, packed_gu: torch.Tensor, offsets: torch.Tensor, I: int,
                               rows: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                               activation: str | None = "silu", out: torch.Tensor | None = None,
                               workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out [R, I] bf16, rows sorted by expert: mxfp4_gated_linear of a[rows[r]] with the weights (and the row of
    `bias` [E, 2I]) of the expert e with offsets[e] <= r < offsets[e+1]. `packed_gu`: mxfp4_prepack_gated_experts';
    `offsets` [E+1] and `rows` [R]: int32 on the device, as mxfp4_moe_route returns them (rows None: row r of `a`).
    Rows of out that belong to no expert are not written."""
    device = a.get_device()
    if device < 0 or device != _device():
        _dev(a, "a")
    st = _raw_stream(device) if stream is None and _raw_stream is not None else _stream(stream)
    tokens, K, lda = _rows_and_stride(a, "a")
    act = ACTIVATIONS.get(activation)
    if act is None:
        _activation(activation)
    if packed_gu.dim() != 2 or not packed_gu.is_contiguous():
        raise ValueError("packed_gu must be a contiguous [E, bytes] buffer (mxfp4_prepack_gated_experts)")
    E = packed_gu.shape[0]
    offsets_ptr = _index(offsets, (E + 1,), a, "offsets")
    if rows is None:
        R, rows_ptr = tokens, None
    else:
        R = rows.shape[0] if rows.dim() == 1 else -1
        rows_ptr = _index(rows, (R,), a, "rows")
    need = 0
    if R and E and I:
        key = ("mxfp4_grouped_gated_linear_workspace_size", mxfp4_prepack_gated_size, device, R, E, I, K)
        known = _SIZES.get(key) or _sizes(key)
        need = known[1]
        if not known[0] or packed_gu.nbytes != E * known[0] or packed_gu.get_device() != device:
            _too_small("packed_gu", f"and exactly {E} * mxfp4_prepack_gated_size({I}, {K})", E * known[0])
    bias_ptr, bias_type = (None, 0) if bias is None else _bias(bias, (E, 2 * I), a)
    if out is None and stream is None and _empty_strided is not None:
        out, ldo = _empty_strided((R, I), (I, 1), _BF16), I
    else:
        out, ldo = _out(out, (R, I), a, "out", stream)
    ws, ws_bytes, _held = _scratch(workspace, need, a, stream, st, device)
    status = load_library().mxfp4_grouped_gated_linear(a.data_ptr(), tokens, K, lda, rows_ptr, offsets_ptr, E,
                                                       packed_gu.data_ptr(), I, bias_ptr, bias_type, act,
                                                       out.data_ptr(), R, ldo, ws, ws_bytes, st)
    if status:
        _check(status, "mxfp4_grouped_gated_linear")
    return out
