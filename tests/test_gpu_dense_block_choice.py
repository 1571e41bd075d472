"""Which kernel runs few rows, by their sizes: of a product, a wavefront alone, through LDS or tiles (the same bits); of the
dense FFN, the gate/up values in fp32 or their codes from the gate/up product (the bits of the three steps)."""
import numpy as np
import pytest
import torch

import dense_block_ref as ref
from block_scaled_fp8xfp4_amd import mxmoe
from dense_block_ref import E2M1, E4M3, codes_like, to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K,fmt,kernel", [
    (1, 4096, 2048, E4M3, "lone16_a8"), (16, 4096, 4096, E2M1, "lone16_a4"), (16, 4096, 4096, E4M3, "rows16_a8"),
    (16, 8192, 576, E4M3, "lone16_a8"), (16, 8192, 1536, E2M1, "lone16_a4"), (9, 16384, 576, E2M1, "lone16_a4"),
    (4, 8192, 1568, E4M3, "rows16_a8"), (16, 16384, 1056, E2M1, "rows16_a4"), (16, 40000, 576, E2M1, "rows16_a4"),
    (16, 32768, 256, E4M3, "rows16_a8"), (8, 4096, 16384, E4M3, "rows16_a8"), (9, 4096, 16384, E4M3, "lone16_a8"),
    (16, 2055, 10240, E4M3, "lone16_a8"), (16, 8192, 16384, E4M3, "lone16_a8"), (16, 8208, 16384, E4M3, "tile"), (16, 4096, 16384, E2M1, "rows16_a4"),
    (17, 4096, 16384, E4M3, "tile"), (17, 96, 64, E4M3, "lone64_a8"), (300, 1030, 96, E2M1, "lone64_a4"),
    (64, 40, 32, E4M3, "lone64_a8"), (16, 1030, 96, E2M1, "lone16_a4")])
def test_product_of_few_rows(M, N, K, fmt, kernel):
    """Short rows are taken by wavefronts alone, and so are rows that do not fit LDS (E4M3 of 9 and more rows at K = 16384;
    as tiles 16 x 4096 x 16384 takes 30 us against 19)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(K)

    def codes(rows, fmt):
        q, sc = codes_like(rows, K, fmt)
        mxmoe.mx_quantize(torch.randn((rows, K), generator=g, device="cuda") * 0.1, q, sc, fmt)
        return q, sc

    a, w = codes(M, fmt), codes(N, E2M1)
    y = torch.full((M + 1, N), float("nan"), device="cuda")
    mxmoe.fp4_block_gemm(*a, fmt, *w, y[:M])
    v = mxmoe.last_variant()
    assert v.startswith("fp4:" + kernel), v
    many = torch.empty((600, N), device="cuda")                       # the same rows in tiles
    mxmoe.fp4_block_gemm(*(t.repeat(-(-600 // M), 1)[:600].contiguous() for t in a), fmt, *w, many)
    assert "tile" in mxmoe.last_variant() or K < 128
    assert torch.equal(y[:M], many[:M]) and torch.isnan(y[M]).all()


@pytest.mark.parametrize("fmt", [E4M3, E2M1])
@pytest.mark.parametrize("T,H,I,values", [
    (1, 8192, 4096, True), (2, 8192, 4096, True), (1, 4096, 2048, True), (4, 4096, 2048, False), (1, 8192, 4128, False),
    (1, 8192, 8192, False), (2, 16384, 8192, False), (1, 4128, 4128, False), (16, 8192, 576, True), (8, 8192, 1056, True),
    (8, 8192, 2048, False), (8, 4096, 576, True), (16, 4096, 576, False), (16, 32, 32, True), (16, 512, 96, True),
    (3, 512, 576, False), (10, 16384, 2048, True), (16, 16384, 1312, True), (16, 16384, 1376, False)])
def test_few_rows(T, H, I, values, fmt):
    """The form with fp32 values up to T * I of about 1.25 H + 1024; past I = 4096 it is 2 to 7 us slower whatever H is."""
    rng = np.random.default_rng(I)
    x, x_sc = (to_dev(t) for t in ref.quantize(ref.activations(rng, T, H), fmt))
    g = torch.Generator(device="cuda")
    g.manual_seed(I)

    def weights(rows, cols):
        q, sc = codes_like(rows, cols, E2M1)
        mxmoe.mx_quantize(torch.randn((rows, cols), generator=g, device="cuda") * 0.02, q, sc, E2M1)
        return q, sc

    w13, w2 = weights(2 * I, H), weights(H, I)
    gu = torch.empty((T, 2 * I), dtype=torch.float32, device="cuda")
    mxmoe.fp4_block_gemm(x, x_sc, fmt, *w13, gu)
    q, sc = codes_like(T, I, fmt)
    mxmoe.mx_swiglu_quantize(gu, q, sc, fmt)
    want, y = (torch.empty((T, H), dtype=torch.float32, device="cuda") for _ in range(2))
    mxmoe.fp4_block_gemm(q, sc, fmt, *w2, want)
    ws = torch.empty(max(256, mxmoe.fp4_dense_ffn_workspace_bytes(T, H, I, fmt)), dtype=torch.uint8, device="cuda")
    mxmoe.fp4_dense_ffn(x, x_sc, fmt, *w13, *w2, fmt, y, ws)
    assert torch.equal(y, want)
    assert (mxmoe.last_variant() == "fp4_ffn:h+") == values, mxmoe.last_variant()
