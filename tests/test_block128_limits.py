"""How many results a block-128 product takes: the limit of the kernel that runs, which is another one where the first choice
does not hold the call.  No operands are given, so a size that is taken ends in MX_EINVAL, one that is not in MX_EUNSUPPORTED."""
import pytest

from block_scaled_fp8xfp4_amd import mxmoe
from block_scaled_fp8xfp4_amd.mxmoe import MX_EINVAL, MX_EUNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    return mxmoe.load()


@pytest.mark.parametrize("M,N,want", [
    (1, 1 << 29, MX_EINVAL), (1, 1 << 30, MX_EINVAL), (16, 1 << 30, MX_EINVAL), (16, (1 << 31) - 64 * 9, MX_EINVAL),
    (17, 1 << 30, MX_EINVAL), (256, (1 << 31) - 256 * 9, MX_EINVAL), (257, (1 << 30) - 4096, MX_EINVAL),
    (1, (1 << 31) - 1, MX_EUNSUPPORTED),                     # 2^25 workgroups of 128 threads
    (1 << 20, 1 << 19, MX_EUNSUPPORTED),                     # 2^23 of 512
    (1 << 20, (1 << 19) - 256, MX_EINVAL)])
@pytest.mark.parametrize("w_rows", [1, 128])
def test_dense_product_sizes(lib, M, N, want, w_rows):
    assert lib.fp8_block128_gemm(None, None, None, None, w_rows, M, N, 16, None, 0, None) == want


@pytest.mark.parametrize("E,R,N,want", [
    (1024, 1024, 1 << 19, MX_EINVAL), (1024, 1024, 1 << 20, MX_EINVAL), (1024, 2048, 1 << 20, MX_EINVAL),   # 16 x 64
    (1024, 2100, 1_200_000, MX_EINVAL), (1024, 20000, 1_000_000, MX_EINVAL),                                # 64 x 128 do not
    (1024, 60000, 1_200_000, MX_EINVAL),                                                                    # nor 128 x 256
    (1024, 1024, 1 << 21, MX_EUNSUPPORTED), (1024, 20000, 1 << 21, MX_EUNSUPPORTED)])
def test_experts_product_sizes(lib, E, R, N, want):
    assert lib.fp8_block128_grouped_gemm(None, None, R, None, None, None, E, N, 16, None, 0, None) == want


@pytest.mark.parametrize("E,N,K,want", [
    (1024, 1 << 14, 127 << 8, MX_EINVAL), (1024, 1 << 15, 1 << 15, MX_EUNSUPPORTED),
    (1024, (1 << 31) - 1, (1 << 31) - 1, MX_EUNSUPPORTED)])      # 2^56 tiles
def test_weight_gradient_sizes(lib, E, N, K, want):
    assert lib.fp8_block128_grouped_wgrad(None, None, None, None, 128, None, E, N, K, None, 0, None) == want
