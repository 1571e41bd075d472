"""Experts' tokens and block-128 products without rows: no tokens, no experts' rows, no expert with rows."""
import numpy as np
import pytest
import torch

from block_scaled_fp8xfp4_amd import mxmoe
from block_scaled_fp8xfp4_amd.layer import ExpertFFN128, ExpertLinear128, FP8Linear128, Route, quantize128, quantize128_t

pytestmark = pytest.mark.gpu
BF16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


def full(value, *shape, dtype=F32):
    return torch.full(shape, value, dtype=dtype, device="cuda")


def test_no_experts_rows():
    x, pos, w = full(1, 3, 40, dtype=BF16), full(0, 3, 2, dtype=I32), full(2, 3, 2)
    none, sc = full(0, 0, 40, dtype=BF16), full(1, 3, 5)
    mxmoe.moe_permute(x, pos, none)
    mxmoe.moe_permute(x, pos, none, sc, full(0, 0, 5))
    y, dw = full(9, 3, 40), full(9, 3, 2)
    mxmoe.moe_unpermute(none, w, pos, y)
    assert (y == 0).all()
    mxmoe.moe_unpermute_grad(x, none, w, pos, full(0, 0, 40, dtype=BF16), dw)
    assert (dw == 0).all()
    mxmoe.moe_unpermute_grad(x, none, w, pos, none)
    mxmoe.moe_unpermute_grad(x, None, w, pos, none)


@pytest.mark.parametrize("rows", [0, 5])
def test_no_expert_has_rows(rows):
    """No rows at all, and rows that are all behind the last expert."""
    off = full(0, 4, dtype=I32)
    layer = ExpertLinear128(*quantize128(full(1, 3, 48, 144), 128), train=True)
    x, g = full(1, rows, 144, dtype=BF16), full(1, rows, 48, dtype=BF16)
    assert layer(x, off).shape == (rows, 48) and layer.input_grad(g, off).shape == (rows, 144)
    for dtype in (F32, BF16):
        assert (layer.weight_grad(g, x, off, dtype=dtype) == 0).all()
    q, sc = quantize128_t(x, off)
    y = full(7, rows, 48)
    mxmoe.fp8_block128_grouped_gemm(*quantize128(x), layer.w, layer.w_sc, off, y)
    assert (y == 7).all() and q.shape[1] == 128 * sc.shape[1]


def test_no_tokens():
    layer = FP8Linear128(*quantize128(full(1, 48, 144), 128), train=True)
    x, g = full(1, 0, 144, dtype=BF16), full(1, 0, 48, dtype=BF16)
    assert layer(x).shape == (0, 48) and layer.input_grad(g).shape == (0, 144) and (layer.weight_grad(g, x) == 0).all()
    route = Route(4, 3, 2)
    route(full(0, 4, 3))
    ffn = ExpertFFN128(*quantize128(full(1, 3, 96, 144), 128), *quantize128(full(1, 3, 144, 48), 128))
    route.slot_pos, route.w = route.slot_pos[:0], route.w[:0]
    route.offsets.zero_()
    assert ffn(x, route).shape == (0, 144)
    assert np.array_equal(route.offsets.cpu().numpy(), np.zeros(4))
