"""The dense block's calls whose operands or results pass 2^32 bytes or 2^31 elements: rows at the far end, bit for bit
those of a small call on the same rows."""
import pytest
import torch

from block_scaled_fp8xfp4_amd import mxmoe
from dense_block_ref import E2M1, E4M3, codes_like

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def codes(rows, K, fmt, seed):
    """Any codes but NaN and scales near 1, made on the GPU."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    q = torch.randint(0, 256, (rows, K if fmt == E4M3 else K // 2), generator=g, dtype=torch.uint8, device="cuda")
    if fmt == E4M3:
        q &= 0xF7                                                     # S.1111.111 is NaN
    return q, torch.randint(120, 134, (rows, K // 32), generator=g, dtype=torch.uint8, device="cuda")


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M,N,K,dtype", [(36000, 65001, 128, BF16),          # 4.7 GB of results, 2.3e9 of them
                                         (270000, 48, 16384, F32),           # 4.4 GB of E4M3 rows
                                         (3, 600000, 16384, F32),            # 4.9 GB of weights
                                         (300, 540000, 16384, BF16),
                                         (16, 140000, 96, F32),
                                         (36000, 65001, 96, BF16)])
@pytest.mark.parametrize("fmt", [E4M3, E2M1])
def test_products(M, N, K, dtype, fmt):
    a, a_sc = codes(M, K, fmt, 1)
    w, w_sc = codes(N, K, E2M1, 2)
    y = torch.empty((M, N), dtype=dtype, device="cuda")
    mxmoe.fp4_block_gemm(a, a_sc, fmt, w, w_sc, y)
    v = mxmoe.last_variant()
    m0, n0 = max(0, M - 9), max(0, N - 64) // 32 * 32
    few = torch.empty((M - m0, N - n0), dtype=dtype, device="cuda")
    cut = [t[m0:].clone() for t in (a, a_sc)], [t[n0:].clone() for t in (w, w_sc)]
    mxmoe.fp4_block_gemm(*cut[0], fmt, *cut[1], few)
    assert torch.equal(y[m0:, n0:], few), v
    first = torch.empty((min(M, 5), min(N, 64)), dtype=dtype, device="cuda")
    cut = [t[:5].clone() for t in (a, a_sc)], [t[:64].clone() for t in (w, w_sc)]
    mxmoe.fp4_block_gemm(*cut[0], fmt, *cut[1], first)
    assert torch.equal(y[:5, :64], first), v


@pytest.mark.parametrize("fmt", [E4M3, E2M1])
def test_ffn(fmt):
    """140000 rows of 16384: 4.6 GB of bf16 results and, in E4M3, 2.3 GB of rows."""
    T, H, I = 140000, 16384, 32
    x, x_sc = codes(T, H, fmt, 3)
    w13, w13_sc = codes(2 * I, H, E2M1, 4)
    w2, w2_sc = codes(H, I, E2M1, 5)
    x_sc -= 7                                                          # gates of a few tens
    w13_sc -= 7

    def ffn(x, x_sc):
        T = x.shape[0]
        y = torch.empty((T, H), dtype=BF16, device="cuda")
        ws = torch.empty(mxmoe.fp4_dense_ffn_workspace_bytes(T, H, I, fmt), dtype=torch.uint8, device="cuda")
        mxmoe.fp4_dense_ffn(x, x_sc, fmt, w13, w13_sc, w2, w2_sc, fmt, y, ws)
        return y

    y = ffn(x, x_sc)
    v = mxmoe.last_variant()
    assert torch.equal(y[-7:], ffn(x[-7:].clone(), x_sc[-7:].clone())), v


@pytest.mark.parametrize("fmt", [E4M3, E2M1])
def test_norm_and_casts(fmt):
    """270000 rows of 8192 elements, 2.2e9 of them; gate/up rows of twice that."""
    T, H = 270000, 8192
    x = torch.randn((T, H), device="cuda", dtype=BF16)
    r = torch.randn((T, H), device="cuda", dtype=F32)
    h, n = torch.empty_like(r), torch.empty((T, H), dtype=BF16, device="cuda")
    q, sc = codes_like(T, H, fmt)

    def small(t):
        return t[-5:].clone()

    mxmoe.mx_add_rmsnorm(x, None, 1e-6, residual=r, h=h, n=n, q=q, sc=sc, fmt=fmt)
    h5, n5 = torch.empty_like(small(h)), torch.empty_like(small(n))
    q5, sc5 = codes_like(5, H, fmt)
    mxmoe.mx_add_rmsnorm(small(x), None, 1e-6, residual=small(r), h=h5, n=n5, q=q5, sc=sc5, fmt=fmt)
    for a, b in ((h, h5), (n, n5), (q, q5), (sc, sc5)):
        assert torch.equal(a[-5:], b)
    del r, h
    mxmoe.mx_dequantize(q, sc, fmt, n)
    mxmoe.mx_dequantize(q5, sc5, fmt, n5)
    assert torch.equal(n[-5:], n5)
    mxmoe.mx_quantize(x, q, sc, fmt)
    mxmoe.mx_quantize(small(x), q5, sc5, fmt)
    assert torch.equal(q[-5:], q5) and torch.equal(sc[-5:], sc5)
    gu = torch.randn((T, 2 * H), device="cuda", dtype=BF16)
    mxmoe.mx_swiglu_quantize(gu, q, sc, fmt)
    mxmoe.mx_swiglu_quantize(small(gu), q5, sc5, fmt)
    assert torch.equal(q[-5:], q5) and torch.equal(sc[-5:], sc5)
