"""Results of more than 64 MB, which go past the caches, at odd widths: vector stores at whatever alignment a row has and the
elements beside them.  What lies there equals the same rows in small calls, and nothing is written past the end."""
import pytest
import torch

from block_scaled_fp8xfp4_amd import mxmoe
from test_gpu_block128_far import codes, scales

pytestmark = pytest.mark.gpu

BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
MIB = 1 << 20


def guarded(rows, cols, dtype):
    """(tensor [rows, cols] of sevens, the whole row's worth that follows it)."""
    flat = torch.full((rows * cols + cols,), 7.0, dtype=dtype, device="cuda")
    return flat[:rows * cols].view(rows, cols), flat[rows * cols:]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("w_rows", [128, 1])
@pytest.mark.parametrize("M,N,K,variant", [(9001, 4099, 272, "tile256x256"), (2050, 17003, 144, "tile256x256"),
                                           (40000, 1001, 48, "tile256x256"), (1150, 40959, 144, "tile128x256"),
                                           (5, 7000009, 16, "tile16x64")])
def test_far_products_of_odd_width(M, N, K, variant, w_rows, dtype):
    a, a_sc, w = codes(M, K), scales(M, -(-K // 128)), codes(N, K)
    w_sc = scales(-(-N // w_rows), -(-K // 128))
    y, behind = guarded(M, N, dtype)
    assert y.nbytes > 64 * MIB
    mxmoe.fp8_block128_gemm(a, a_sc, w, w_sc, y)
    assert mxmoe.last_variant() == "b128:" + variant
    step = 40 if N < 10**5 else 1
    for r in (0, M // 2, M - step):
        z = torch.empty((step, N), dtype=dtype, device="cuda")
        mxmoe.fp8_block128_gemm(a[r:r + step].contiguous(), a_sc[r:r + step].contiguous(), w, w_sc, z)
        assert torch.equal(y[r:r + step], z), r
    assert (behind == 7).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("E,per,N,K,variant", [(20, 1000, 2051, 144, "tile256x256"), (16, 60, 35101, 144, "tile128x256"),
                                               (256, 30, 4501, 144, "tile64x128"), (300, 20, 5701, 2064, "tile64x64"),
                                               (300, 2, 60007, 144, "tile16x64")])
def test_far_experts_of_odd_width(E, per, N, K, variant, dtype):
    R, nb = E * per, -(-K // 128)
    a, a_sc, w, w_sc = codes(R, K), scales(R, nb), codes(E, N, K), scales(E, -(-N // 128), nb)
    off = (torch.arange(E + 1, device="cuda") * per).int()
    y, behind = guarded(R, N, dtype)
    assert y.nbytes > 64 * MIB
    mxmoe.fp8_block128_grouped_gemm(a, a_sc, w, w_sc, off, y)
    assert mxmoe.last_variant() == "b128:" + variant
    for e in (0, 1, E // 2, E - 1):
        z = torch.empty((per, N), dtype=dtype, device="cuda")
        s = slice(e * per, (e + 1) * per)
        mxmoe.fp8_block128_gemm(a[s].contiguous(), a_sc[s].contiguous(), w[e], w_sc[e], z)
        assert torch.equal(y[s], z), e
    assert (behind == 7).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("E,N,K", [(40, 1001, 1021), (9, 5003, 1001), (300, 130, 1999)])
def test_far_weight_gradients_of_odd_width(E, N, K, dtype):
    per = 100
    ld = mxmoe.fp8_quantize128_t_cols(E * per, E)
    a, a_sc, b, b_sc = codes(N, ld), scales(N, ld // 128), codes(K, ld), scales(K, ld // 128)
    off = (torch.arange(E + 1, device="cuda") * per).int()
    flat, behind = guarded(E * N, K, dtype)
    dw = flat.view(E, N, K)
    assert dw.nbytes > 64 * MIB
    mxmoe.fp8_block128_grouped_wgrad(a, a_sc, b, b_sc, off, dw)
    for e in (0, 1, E // 2, E - 1):
        s = slice(e * 128, (e + 1) * 128)
        z = torch.empty((N, K), dtype=dtype, device="cuda")
        mxmoe.fp8_block128_gemm(a[:, s].contiguous(), a_sc[:, e:e + 1].contiguous(), b[:, s].contiguous(),
                                b_sc[:, e:e + 1].contiguous(), z)
        assert torch.equal(dw[e], z), e
    assert (behind == 7).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H", [2051, 4104, 9])
def test_far_tokens_of_odd_width(dtype, H):
    T, k = 80 * MIB // (H * dtype.itemsize * 4) + 1, 4
    x, w = torch.randn((T, H), device="cuda").to(dtype), torch.rand((T, k), device="cuda")
    pos = torch.randperm(T * k, device="cuda").int().view(T, k)
    out, behind = guarded(T * k, H, dtype)
    assert out.nbytes > 64 * MIB
    mxmoe.moe_permute(x, pos, out)
    assert torch.equal(out[pos.long()], x[:, None].expand(T, k, H)) and (behind == 7).all()
    part = torch.arange(0, T, max(1, T // 500), device="cuda")       # these tokens by themselves are 64 MB and less
    mine, few_pos = out[pos[part].long()].view(-1, H), torch.arange(len(part) * k, dtype=torch.int32, device="cuda").view(-1, k)
    few_weights = w[part].contiguous()
    assert mine.nbytes <= 64 * MIB
    for y_type in (BF16, F32):
        y, after = guarded(T, H, y_type)
        mxmoe.moe_unpermute(out, w, pos, y)
        few = torch.empty((len(part), H), dtype=y_type, device="cuda")
        mxmoe.moe_unpermute(mine, few_weights, few_pos, few)
        assert torch.equal(y[part], few) and (after == 7).all()
    dy, (d_o, after) = torch.randn((T, H), device="cuda").to(dtype), guarded(T * k, H, dtype)
    dw = torch.empty_like(w)
    mxmoe.moe_unpermute_grad(dy, out, w, pos, d_o, dw)
    assert torch.equal(d_o[pos.long()], (dy[:, None].float() * w[:, :, None]).to(dtype)) and (after == 7).all()
    few_o, few_w = torch.empty_like(mine), torch.empty_like(few_weights)
    mxmoe.moe_unpermute_grad(dy[part].contiguous(), mine, few_weights, few_pos, few_o, few_w)
    assert torch.equal(few_w, dw[part]) and torch.equal(few_o, d_o[pos[part].long()].view(-1, H))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols,groups", [(40000, 1100, 64), (66000, 570, 0), (300000, 129, 300), (128 * 1400, 192, 0)])
def test_columns_of_many_tiles(dtype, rows, cols, groups):
    """Two column tiles to a workgroup, the last one alone or partly there, with groups and without: the columns by themselves."""
    src = torch.randn((rows, cols), device="cuda").to(dtype)
    src[:, ::7] *= 30
    off = None
    if groups:
        cut = torch.sort(torch.randint(0, rows + 1, (groups - 1,), device="cuda")).values
        off = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), rows)]).int()
    ld = mxmoe.fp8_quantize128_t_cols(rows, max(groups, 1))
    assert ld // 128 * -(-cols // 64) > 4096
    q, sc = torch.full((cols, ld), 0xA5, dtype=U8, device="cuda"), torch.full((cols, ld // 128), -7.0, device="cuda")
    mxmoe.fp8_quantize128_t(src, q, sc, off)
    for c in (0, 60, cols // 128 * 128 - 4, cols - 5):
        q1, sc1 = torch.full((5, ld), 0xA5, dtype=U8, device="cuda"), torch.full((5, ld // 128), -7.0, device="cuda")
        mxmoe.fp8_quantize128_t(src[:, c:c + 5].contiguous(), q1, sc1, off)
        assert torch.equal(q[c:c + 5], q1) and torch.equal(sc[c:c + 5], sc1), c
