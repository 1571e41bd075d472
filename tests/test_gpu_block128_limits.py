"""Products of so many columns that the kernel of few rows, or of small experts, is not the one that a launch holds: the same
bits as the columns by themselves."""
import pytest
import torch

from block_scaled_fp8xfp4_amd import mxmoe

pytestmark = pytest.mark.gpu

BF16, U8, K = torch.bfloat16, torch.uint8, 16


def codes(*shape):
    return torch.randint(0, 0x70, shape, dtype=U8, device="cuda")


def scales(*shape):
    return torch.rand(shape, device="cuda") * 1e-2 + 1e-3


def columns(a, a_sc, w, w_sc, n0):
    """The product with 256 columns from n0 on, a multiple of 128."""
    n = min(256, w.shape[0] - n0)
    y = torch.empty((a.shape[0], n), dtype=BF16, device="cuda")
    mxmoe.fp8_block128_gemm(a, a_sc, w[n0:n0 + n].contiguous(), w_sc[n0 // 128:n0 // 128 + 2].contiguous(), y)
    return y


def test_one_row_of_more_than_2_29_columns():
    N = (1 << 29) + 1000
    a, a_sc, w, w_sc = codes(1, K), scales(1, 1), codes(N, K), scales(-(-N // 128), 1)
    y = torch.empty((1, N), dtype=BF16, device="cuda")
    mxmoe.fp8_block128_gemm(a, a_sc, w, w_sc, y)
    assert mxmoe.last_variant() == "b128:tile16x64"
    for n0 in (0, 1 << 28, (1 << 29) - 128, N // 128 * 128):
        assert torch.equal(y[:, n0:n0 + 256], columns(a, a_sc, w, w_sc, n0)), n0


@pytest.mark.parametrize("E,R,N,variant", [(1024, 1024, (1 << 19) + 200, "tile16x64"), (1024, 2100, (1 << 20) + 50000, "tile128x256")])
def test_experts_of_more_than_2_19_columns(E, R, N, variant):
    a, a_sc, w, w_sc = codes(R, K), scales(R, 1), codes(E, N, K), scales(E, -(-N // 128), 1)
    off = (torch.arange(E + 1) * R // E).int().cuda()
    y = torch.empty((R, N), dtype=BF16, device="cuda")
    mxmoe.fp8_block128_grouped_gemm(a, a_sc, w, w_sc, off, y)
    assert mxmoe.last_variant() == "b128:" + variant
    off = off.tolist()
    for e in (0, 500, E - 1):
        i, j = off[e], off[e + 1]
        for n0 in (0, 1 << 18, N // 128 * 128):
            assert torch.equal(y[i:j, n0:n0 + 256], columns(a[i:j].contiguous(), a_sc[i:j].contiguous(), w[e], w_sc[e], n0)), (e, n0)
