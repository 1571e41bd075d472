"""The experts' tokens and FP8 products past 2^32 bytes and 2^31 elements: what lies far equals the same rows by themselves."""
import pytest
import torch

from block_scaled_fp8xfp4_amd import mxmoe

pytestmark = pytest.mark.gpu

BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


def codes(*shape):
    return torch.randint(0, 0x70, shape, dtype=U8, device="cuda")


def scales(*shape):
    return torch.rand(shape, device="cuda") * 1e-2 + 1e-3


def test_product_with_far_results_and_rows():
    M, N, K = 70000, 33000, 128
    a, a_sc, w, w_sc = codes(M, K), scales(M, 1), codes(N, K), scales(-(-N // 128), 1)
    y = torch.empty((M, N), dtype=BF16, device="cuda")
    mxmoe.fp8_block128_gemm(a, a_sc, w, w_sc, y)
    for r in (0, 65070, M - 40):                       # the second: where elements pass 2^31
        z = torch.empty((40, N), dtype=BF16, device="cuda")
        mxmoe.fp8_block128_gemm(a[r:r + 40].contiguous(), a_sc[r:r + 40].contiguous(), w, w_sc, z)
        assert torch.equal(y[r:r + 40], z)


def test_product_with_far_operands():
    M, N, K = 300000, 200, 16384
    a, a_sc, w, w_sc = codes(M, K), scales(M, K // 128), codes(N, K), scales(2, K // 128)
    y = torch.empty((M, N), dtype=F32, device="cuda")
    mxmoe.fp8_block128_gemm(a, a_sc, w, w_sc, y)
    for r in (0, 262144 - 20, M - 40):
        z = torch.empty((40, N), dtype=F32, device="cuda")
        mxmoe.fp8_block128_gemm(a[r:r + 40].contiguous(), a_sc[r:r + 40].contiguous(), w, w_sc, z)
        assert torch.equal(y[r:r + 40], z)


@pytest.mark.parametrize("per", [1, 40, 150])
def test_experts_with_far_weights(per):
    E, N, K = 300, 4096, 4096
    w, w_sc = codes(E, N, K), scales(E, N // 128, K // 128)
    R = E * per
    a, a_sc = codes(R, K), scales(R, K // 128)
    off = (torch.arange(E + 1, device="cuda") * per).int()
    y = torch.empty((R, N), dtype=BF16, device="cuda")
    mxmoe.fp8_block128_grouped_gemm(a, a_sc, w, w_sc, off, y)
    for e in (0, 127, 128, 255, 256, E - 1):
        z = torch.empty((per, N), dtype=BF16, device="cuda")
        mxmoe.fp8_block128_gemm(a[e * per:(e + 1) * per].contiguous(), a_sc[e * per:(e + 1) * per].contiguous(), w[e], w_sc[e], z)
        assert torch.equal(y[e * per:(e + 1) * per], z)


def test_far_weight_gradients():
    E, N, K, per = 300, 2048, 4096, 100
    ld = mxmoe.fp8_quantize128_t_cols(E * per, E)
    a, a_sc, b, b_sc = codes(N, ld), scales(N, ld // 128), codes(K, ld), scales(K, ld // 128)
    off = (torch.arange(E + 1, device="cuda") * per).int()
    dw = torch.empty((E, N, K), dtype=BF16, device="cuda")
    mxmoe.fp8_block128_grouped_wgrad(a, a_sc, b, b_sc, off, dw)
    for e in (0, 255, 256, E - 1):
        z = torch.empty((N, K), dtype=BF16, device="cuda")
        mxmoe.fp8_block128_gemm(a[:, e * 128:(e + 1) * 128].contiguous(), a_sc[:, e:e + 1].contiguous(),
                                b[:, e * 128:(e + 1) * 128].contiguous(), b_sc[:, e:e + 1].contiguous(), z)
        assert torch.equal(dw[e], z)


def test_far_tokens():
    T, k, H = 70000, 8, 8192
    x = torch.randn((T, H), device="cuda").to(BF16)
    pos = torch.randperm(T * k, device="cuda").int().view(T, k)
    out = torch.empty((T * k, H), dtype=BF16, device="cuda")          # 9.2 GB
    mxmoe.moe_permute(x, pos, out)
    back = torch.argsort(pos.view(-1))
    for p in (0, 262143, 262144, T * k - 1):
        assert torch.equal(out[p], x[int(back[p]) // k])
    y = torch.empty((T, H), device="cuda")
    mxmoe.moe_unpermute(out, None, pos, y)
    assert torch.equal(y, x.float() * k)                               # eight times the same bf16 value: exact
    w = torch.rand((T, k), device="cuda")
    dw = torch.empty_like(w)
    mxmoe.moe_unpermute_grad(x, out, w, pos, out, dw)
    for p in (0, 262144, T * k - 1):
        t, j = divmod(int(back[p]), k)
        assert torch.equal(out[p], (x[t].float() * float(w[t, j])).to(BF16))
    norms = x.double().square().sum(-1)
    assert ((dw.double() - norms[:, None]).abs() <= 2e-5 * norms[:, None]).all()   # (128 + 7) 2^-24 of a sum of squares


def test_far_casts():
    rows, cols = 600000, 4096
    src = torch.randn((rows, cols), device="cuda", dtype=BF16)         # 4.9 GB
    q, sc = torch.empty((rows, cols), dtype=U8, device="cuda"), torch.empty((rows, cols // 128), device="cuda")
    mxmoe.fp8_quantize128(src, q, sc)
    for r in (0, 524287, 524288, rows - 3):
        q1, sc1 = torch.empty((3, cols), dtype=U8, device="cuda"), torch.empty((3, cols // 128), device="cuda")
        mxmoe.fp8_quantize128(src[r:r + 3], q1, sc1)
        assert torch.equal(q[r:r + 3], q1) and torch.equal(sc[r:r + 3], sc1)
    gu = src.view(rows, cols)
    q2, sc2 = torch.empty((rows, cols // 2), dtype=U8, device="cuda"), torch.empty((rows, cols // 256), device="cuda")
    mxmoe.fp8_swiglu_quantize128(gu, q2, sc2)
    q1, sc1 = torch.empty((3, cols // 2), dtype=U8, device="cuda"), torch.empty((3, cols // 256), device="cuda")
    mxmoe.fp8_swiglu_quantize128(gu[-3:], q1, sc1)
    assert torch.equal(q2[-3:], q1) and torch.equal(sc2[-3:], sc1)
    del q2, sc2
    ld = mxmoe.fp8_quantize128_t_cols(rows)
    qt, sct = torch.empty((cols, ld), dtype=U8, device="cuda"), torch.empty((cols, ld // 128), device="cuda")
    mxmoe.fp8_quantize128_t(src, qt, sct)
    part = src[-(rows % 128 or 128):].contiguous()
    n = part.shape[0]
    q1, sc1 = torch.empty((cols, 128), dtype=U8, device="cuda"), torch.empty((cols, 1), device="cuda")
    mxmoe.fp8_quantize128_t(part, q1, sc1)
    assert n > 0 and torch.equal(qt[:, -128:], q1) and torch.equal(sct[:, -1:], sc1)
    tq, tsc = torch.empty((rows, cols), dtype=U8, device="cuda"), torch.empty((-(-rows // 128), cols // 128), device="cuda")
    mxmoe.fp8_quantize128(src, tq, tsc, 128)
    q1, sc1 = torch.empty((n, cols), dtype=U8, device="cuda"), torch.empty((1, cols // 128), device="cuda")
    mxmoe.fp8_quantize128(part, q1, sc1, 128)
    assert torch.equal(tq[-n:], q1) and torch.equal(tsc[-1:], sc1)
