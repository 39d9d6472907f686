"""The binding remembers the sizes that the library answers by shape, but not without end: a process that meets ever
new lengths of prompts holds a bounded number of them, and a size that was dropped is asked for again."""
import torch

import block_scaled_mxfp4_bf16_gb300 as mx
from block_scaled_mxfp4_bf16_gb300 import linear, moe
from test_binding_checks import dev
from test_linear_checks import bf16, gated_packed, i32, lib, packed, ws  # noqa: F401  (lib: the fixture)

TABLES = {"gemm workspace": lambda: mx._WS_NEED, "packed": lambda: mx._PACKED_NEED, "experts": lambda: moe._NEED,
          "epilogue": lambda: linear._SIZES}


def test_tables_of_sizes_are_bounded(lib):  # noqa: F811
    limit = mx._REMEMBERED
    assert 1000 <= limit <= 1 << 16
    dense, gu, experts, x = packed(1, 128, 256)[0], gated_packed(1, 64, 256), packed(1, 128, 256), bf16(2 * limit, 256)
    offsets = i32(0, 1)
    wide = dev(torch.zeros(1 << 22, dtype=torch.uint8))
    for M in range(1, limit + 40):
        mx.mxfp4_linear(x[:M], dense, 128, out=bf16(M, 128), workspace=ws(), stream=0)
        mx._ws_need(x.device, M, 128, 256)
        moe._need("mxfp4_grouped_gemm_workspace_size", -1, M, 1, 128, 256)
        mx._check_packed(wide, M, 256, None)
    mx.mxfp4_gated_linear(x[:3], gu[0], 64, out=bf16(3, 64), workspace=ws(), stream=0)
    mx.mxfp4_grouped_gemm(x[:1], experts, offsets, 128, c=bf16(1, 128), workspace=ws(), stream=0)
    for name, table in TABLES.items():
        assert 1 <= len(table()) <= limit, name


def test_a_size_of_the_epilogue_products_is_kept_once(lib):  # noqa: F811
    before = len(moe._NEED)
    mx.mxfp4_linear(bf16(7, 256), packed(1, 128, 256)[0], 128, out=bf16(7, 128), workspace=ws(), stream=0)
    assert len(linear._SIZES) == 1 and len(moe._NEED) == before
