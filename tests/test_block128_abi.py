"""The entry points of the experts' tokens and of FP8 products with a scale for each block of 128 refuse bad arguments on the
host, before any HIP call: status codes of the C-ABI, ValueErrors of the binding."""
import ctypes
import os

import pytest
import torch

from block_scaled_fp8xfp4_amd import mxmoe
from block_scaled_fp8xfp4_amd.mxmoe import MX_EINVAL, MX_EUNSUPPORTED, MX_OK

FAKE = ctypes.c_void_p(1 << 20)        # aligned, never dereferenced: validation fails first
ODD = ctypes.c_void_p((1 << 20) + 2)
BYTE = ctypes.c_void_p((1 << 20) + 1)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mxmoe.LIB_PATH):
        import block_scaled_fp8xfp4_amd.build as b
        b.build()
    return mxmoe.load()


def test_permute_rejects_bad_arguments(lib):
    def call(x=FAKE, ld=64, row=64, xs=FAKE, sc=8, pos=FAKE, T=4, k=2, out=FAKE, os_=FAKE, R=8):
        return lib.moe_permute(x, ld, row, xs, sc, pos, T, k, out, os_, R, None)
    for bad in (dict(T=-1), dict(k=0), dict(k=17), dict(row=0), dict(sc=-1), dict(ld=63), dict(R=-1), dict(x=None),
                dict(pos=None), dict(out=None), dict(xs=None), dict(os_=None), dict(pos=ODD)):
        assert call(**bad) == MX_EINVAL, bad
    assert call(T=1 << 30) == MX_EUNSUPPORTED and call(row=1 << 41, ld=1 << 41) == MX_EUNSUPPORTED
    assert call(R=1 << 60) == MX_EUNSUPPORTED and call(ld=1 << 59) == MX_EUNSUPPORTED
    assert call(T=0, x=None, pos=None, out=None, xs=None, os_=None) == MX_OK


def test_unpermute_rejects_bad_arguments(lib):
    def call(o=FAKE, ot=1, R=8, w=FAKE, pos=FAKE, T=4, k=2, H=64, y=FAKE, yt=0):
        return lib.moe_unpermute(o, ot, R, w, pos, T, k, H, y, yt, None)
    for bad in (dict(T=-1), dict(k=0), dict(k=17), dict(H=0), dict(R=-1), dict(ot=2), dict(yt=2), dict(o=None), dict(pos=None),
                dict(y=None), dict(o=BYTE), dict(o=ODD, ot=0), dict(w=ODD), dict(pos=ODD), dict(y=BYTE), dict(y=ODD, yt=1)):
        assert call(**bad) == MX_EINVAL, bad
    assert call(T=1 << 26, k=16, H=16) == MX_EUNSUPPORTED and call(T=1 << 20, H=1 << 12) == MX_EUNSUPPORTED
    assert call(R=1 << 60) == MX_EUNSUPPORTED
    assert call(T=0, o=None, w=None, pos=None, y=None) == MX_OK


def test_unpermute_grad_rejects_bad_arguments(lib):
    def call(dy=FAKE, dt=1, o=FAKE, ot=1, R=8, w=FAKE, pos=FAKE, T=4, k=2, H=64, d=FAKE, dw=FAKE):
        return lib.moe_unpermute_grad(dy, dt, o, ot, R, w, pos, T, k, H, d, dw, None)
    for bad in (dict(T=-1), dict(k=0), dict(k=17), dict(H=0), dict(R=-1), dict(ot=2), dict(dt=-1), dict(dy=None), dict(o=None),
                dict(pos=None), dict(d=None, dw=None), dict(dy=BYTE), dict(dy=ODD, dt=0), dict(o=BYTE), dict(d=BYTE),
                dict(d=ODD, ot=0), dict(dw=ODD), dict(w=ODD), dict(pos=ODD)):
        assert call(**bad) == MX_EINVAL, bad
    assert call(T=1 << 24, k=2, H=16) == MX_EUNSUPPORTED
    assert call(T=0, dy=None, o=None, w=None, pos=None, d=None, dw=None) == MX_OK


def test_tokens_columns_stay_below_2_31(lib):
    """Rows of more than 2^30 columns, whose last pieces an int would not hold, and calls without experts' rows."""
    H = (1 << 30) + 1
    assert lib.moe_unpermute(FAKE, 1, 1, None, FAKE, 1, 1, H, FAKE, 0, None) == MX_EUNSUPPORTED
    assert lib.moe_unpermute_grad(FAKE, 1, FAKE, 1, 1, None, FAKE, 1, 1, H, FAKE, None, None) == MX_EUNSUPPORTED
    assert lib.moe_permute(FAKE, 64, 64, None, 0, FAKE, 4, 2, None, None, 0, None) == MX_OK
    assert lib.moe_unpermute_grad(FAKE, 1, None, 1, 0, None, FAKE, 4, 2, 64, None, None, None) == MX_OK


def test_quantize_rejects_bad_arguments(lib):
    def call(src=FAKE, dt=1, ld=64, n=2, rows=4, cols=64, br=1, q=FAKE, sc=FAKE):
        return lib.fp8_quantize128(src, dt, ld, n, rows, cols, br, q, sc, None)
    for bad in (dict(n=-1), dict(rows=-1), dict(cols=0), dict(cols=24), dict(dt=2), dict(br=2), dict(br=0), dict(ld=48),
                dict(ld=68), dict(dt=0, ld=66), dict(src=None), dict(q=None), dict(sc=None), dict(src=ODD), dict(q=ODD),
                dict(sc=ODD)):
        assert call(**bad) == MX_EINVAL, bad
    assert call(rows=1 << 28) == MX_EUNSUPPORTED and call(rows=1 << 40) == MX_EUNSUPPORTED
    assert call(br=128, rows=1 << 31) == MX_EUNSUPPORTED and call(ld=1 << 58) == MX_EUNSUPPORTED
    assert call(n=0, src=None, q=None, sc=None) == MX_OK and call(rows=0, src=None, q=None, sc=None) == MX_OK


def test_swiglu_quantize_rejects_bad_arguments(lib):
    def call(gu=FAKE, dt=0, ld=128, T=4, I=64, q=FAKE, sc=FAKE):
        return lib.fp8_swiglu_quantize128(gu, dt, ld, T, I, q, sc, None)
    for bad in (dict(T=-1), dict(I=0), dict(I=24), dict(dt=2), dict(ld=127), dict(ld=130), dict(dt=1, ld=132), dict(gu=None),
                dict(q=None), dict(sc=None), dict(gu=ODD), dict(q=ODD), dict(sc=ODD)):
        assert call(**bad) == MX_EINVAL, bad
    assert call(T=1 << 28) == MX_EUNSUPPORTED and call(T=0, gu=None, q=None, sc=None) == MX_OK


def test_quantize_columns_rejects_bad_arguments(lib):
    def call(src=FAKE, dt=1, ld=64, rows=200, cols=64, off=FAKE, E=3, q=FAKE, sc=FAKE, q_ld=512):
        return lib.fp8_quantize128_t(src, dt, ld, rows, cols, off, E, q, sc, q_ld, None)
    for bad in (dict(rows=-1), dict(cols=0), dict(dt=2), dict(ld=63), dict(E=0), dict(E=1025), dict(off=None), dict(q_ld=500),
                dict(q_ld=384), dict(rows=1 << 31, q_ld=1 << 33), dict(src=None), dict(q=None), dict(sc=None), dict(src=BYTE),
                dict(src=ODD, dt=0), dict(off=ODD), dict(q=ODD), dict(sc=ODD)):
        assert call(**bad) == MX_EINVAL, bad
    assert call(rows=1 << 30, cols=1 << 12, ld=1 << 12, q_ld=1 << 31) == MX_EUNSUPPORTED
    assert call(rows=0, src=None, q=None, sc=None, q_ld=0) == MX_OK


def test_columns_hold_any_split():
    for rows in (0, 1, 5, 127, 128, 129, 300, 1000):
        for E in (1, 2, 3, 7, 300):
            worst = 0
            for a in range(min(E, 40)):
                # as many groups of one row as there are, the rest in one group; and rows just past a block
                ones = min(a, rows)
                worst = max(worst, ones * 128 + -(-(rows - ones) // 128) * 128)
                cut = min(a, rows // 129)
                worst = max(worst, cut * 256 + -(-(rows - cut * 129) // 128) * 128)
            assert mxmoe.fp8_quantize128_t_cols(rows, E) >= worst, (rows, E)
    assert mxmoe.fp8_quantize128_t_cols(-1, 1) == 0 and mxmoe.fp8_quantize128_t_cols(5, 0) == 0


def test_product_rejects_bad_arguments(lib):
    def call(a=FAKE, a_sc=FAKE, w=FAKE, w_sc=FAKE, wr=128, M=4, N=5, K=144, y=FAKE, dt=0):
        return lib.fp8_block128_gemm(a, a_sc, w, w_sc, wr, M, N, K, y, dt, None)
    for bad in (dict(M=-1), dict(N=0), dict(K=0), dict(K=24), dict(wr=0), dict(wr=64), dict(dt=2), dict(a=None), dict(a_sc=None),
                dict(w=None), dict(w_sc=None), dict(y=None), dict(a=ODD), dict(w=ODD), dict(a_sc=ODD), dict(w_sc=ODD),
                dict(y=BYTE), dict(y=ODD, dt=1)):
        assert call(**bad) == MX_EINVAL, bad
    assert call(K=(1 << 23) + 16) == MX_EUNSUPPORTED
    assert call(M=(1 << 31) - 1, N=(1 << 31) - 1) == MX_EUNSUPPORTED
    assert call(M=0, a=None, a_sc=None, w=None, w_sc=None, y=None) == MX_OK


def test_grouped_product_rejects_bad_arguments(lib):
    def call(a=FAKE, a_sc=FAKE, R=4, w=FAKE, w_sc=FAKE, off=FAKE, E=3, N=5, K=144, y=FAKE, dt=0):
        return lib.fp8_block128_grouped_gemm(a, a_sc, R, w, w_sc, off, E, N, K, y, dt, None)
    for bad in (dict(R=-1), dict(E=0), dict(E=1025), dict(N=0), dict(K=0), dict(K=24), dict(dt=2), dict(a=None), dict(a_sc=None),
                dict(w=None), dict(w_sc=None), dict(off=None), dict(y=None), dict(a=ODD), dict(w=ODD), dict(a_sc=ODD),
                dict(w_sc=ODD), dict(off=ODD), dict(y=BYTE), dict(y=ODD, dt=1)):
        assert call(**bad) == MX_EINVAL, bad
    assert call(K=(1 << 23) + 16) == MX_EUNSUPPORTED and call(R=(1 << 31) - 1, N=(1 << 31) - 1) == MX_EUNSUPPORTED
    assert call(R=0, a=None, a_sc=None, w=None, w_sc=None, off=None, y=None) == MX_OK


def test_grouped_wgrad_rejects_bad_arguments(lib):
    def call(a=FAKE, a_sc=FAKE, b=FAKE, b_sc=FAKE, ld=512, off=FAKE, E=3, N=5, K=7, dw=FAKE, dt=0):
        return lib.fp8_block128_grouped_wgrad(a, a_sc, b, b_sc, ld, off, E, N, K, dw, dt, None)
    for bad in (dict(ld=-128), dict(ld=500), dict(E=0), dict(E=1025), dict(N=0), dict(K=0), dict(dt=2), dict(a=None),
                dict(a_sc=None), dict(b=None), dict(b_sc=None), dict(off=None), dict(dw=None), dict(a=ODD), dict(b=ODD),
                dict(a_sc=ODD), dict(b_sc=ODD), dict(off=ODD), dict(dw=BYTE), dict(dw=ODD, dt=1)):
        assert call(**bad) == MX_EINVAL, bad
    assert call(ld=(1 << 23) + 128) == MX_EUNSUPPORTED and call(N=(1 << 31) - 1, K=(1 << 31) - 1) == MX_EUNSUPPORTED


def u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


def f32(*s):
    return torch.zeros(s, dtype=torch.float32)


def bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


@pytest.mark.parametrize("call", [
    lambda: mxmoe.moe_permute(bf(64), i32(2, 2), bf(4, 64)),
    lambda: mxmoe.moe_permute(bf(2, 64), i32(2, 2), f32(4, 64)),
    lambda: mxmoe.moe_permute(bf(2, 64), i32(2, 2), bf(4, 32)),
    lambda: mxmoe.moe_permute(bf(2, 64), i32(3, 2), bf(4, 64)),
    lambda: mxmoe.moe_permute(bf(2, 64), i32(2, 2).long(), bf(4, 64)),
    lambda: mxmoe.moe_permute(bf(64, 2).t(), i32(2, 2), bf(4, 64)),
    lambda: mxmoe.moe_permute(bf(2, 64), i32(2, 2), bf(4, 128)[:, :64]),
    lambda: mxmoe.moe_permute(bf(2, 64), i32(2, 2), bf(4, 64), f32(2, 1)),
    lambda: mxmoe.moe_permute(bf(2, 64), i32(2, 2), bf(4, 64), f32(2, 1), f32(3, 1)),
    lambda: mxmoe.moe_permute(bf(2, 64), i32(2, 2), bf(4, 64), f32(2, 1), u8(4, 1)),
    lambda: mxmoe.moe_permute(bf(2, 0), i32(2, 2), bf(4, 0)),
    lambda: mxmoe.moe_permute(bf(2, 64), i32(2, 2), bf(4, 64)),                      # not on the current device
    lambda: mxmoe.moe_unpermute(bf(4, 64).half(), None, i32(2, 2), bf(2, 64)),
    lambda: mxmoe.moe_unpermute(bf(4, 64), bf(2, 2), i32(2, 2), bf(2, 64)),
    lambda: mxmoe.moe_unpermute(bf(4, 64), f32(2, 3), i32(2, 2), bf(2, 64)),
    lambda: mxmoe.moe_unpermute(bf(4, 64), None, i32(3, 2), bf(2, 64)),
    lambda: mxmoe.moe_unpermute(bf(4, 64), None, i32(2, 2), bf(2, 32)),
    lambda: mxmoe.moe_unpermute(bf(4, 128)[:, :64], None, i32(2, 2), bf(2, 64)),
    lambda: mxmoe.moe_unpermute_grad(bf(2, 64), None, None, i32(2, 2)),
    lambda: mxmoe.moe_unpermute_grad(bf(2, 64), None, None, i32(2, 2), dw=f32(2, 2)),
    lambda: mxmoe.moe_unpermute_grad(bf(2, 64), None, None, i32(2, 2), bf(4, 64), f32(2, 2)),
    lambda: mxmoe.moe_unpermute_grad(bf(2, 64), bf(4, 64), None, i32(2, 2), f32(4, 64)),
    lambda: mxmoe.moe_unpermute_grad(bf(2, 64), bf(4, 32), None, i32(2, 2), bf(4, 32)),
    lambda: mxmoe.moe_unpermute_grad(bf(2, 64), bf(4, 64), None, i32(2, 2), bf(4, 64), bf(2, 2)),
    lambda: mxmoe.fp8_quantize128(bf(64), u8(64), f32(1)),
    lambda: mxmoe.fp8_quantize128(bf(2, 64), u8(2, 64), f32(2, 1), 64),
    lambda: mxmoe.fp8_quantize128(bf(2, 64).half(), u8(2, 64), f32(2, 1)),
    lambda: mxmoe.fp8_quantize128(bf(2, 144), u8(2, 144), f32(2, 1)),
    lambda: mxmoe.fp8_quantize128(bf(2, 144), u8(2, 144), f32(2, 2), 128),
    lambda: mxmoe.fp8_quantize128(bf(3, 2, 144).transpose(0, 1), u8(2, 3, 144), f32(2, 3, 2)),
    lambda: mxmoe.fp8_swiglu_quantize128(bf(2, 63), u8(2, 31), f32(2, 1)),
    lambda: mxmoe.fp8_swiglu_quantize128(bf(2, 64), u8(2, 64), f32(2, 1)),
    lambda: mxmoe.fp8_swiglu_quantize128(bf(2, 64), u8(2, 32), u8(2, 1)),
    lambda: mxmoe.fp8_quantize128_t(bf(200, 64), u8(64, 200), f32(64, 2)),
    lambda: mxmoe.fp8_quantize128_t(bf(200, 64), u8(32, 256), f32(64, 2)),
    lambda: mxmoe.fp8_quantize128_t(bf(200, 64), u8(64, 256), f32(64, 1)),
    lambda: mxmoe.fp8_quantize128_t(bf(200, 64), u8(64, 512), f32(64, 4), torch.zeros(4)),
    lambda: mxmoe.fp8_quantize128_t(bf(64, 200).t(), u8(64, 256), f32(64, 2)),
    lambda: mxmoe.fp8_block128_gemm(u8(4, 256), f32(4, 2), u8(8, 256), f32(2, 2), bf(4, 8)),
    lambda: mxmoe.fp8_block128_gemm(u8(4, 256), f32(4, 2), u8(8, 256), f32(1, 2), bf(4, 9)),
    lambda: mxmoe.fp8_block128_gemm(u8(4, 256), f32(4, 1), u8(8, 256), f32(1, 2), bf(4, 8)),
    lambda: mxmoe.fp8_block128_gemm(u8(4, 128), f32(4, 2), u8(8, 256), f32(1, 2), bf(4, 8)),
    lambda: mxmoe.fp8_block128_gemm(u8(4, 256), f32(4, 2), u8(8, 256), f32(1, 2), bf(4, 8).half()),
    lambda: mxmoe.fp8_block128_gemm(u8(4, 256), u8(4, 2), u8(8, 256), f32(1, 2), bf(4, 8)),
    lambda: mxmoe.fp8_block128_grouped_gemm(u8(4, 256), f32(4, 2), u8(8, 256), f32(1, 2), i32(4), bf(4, 8)),
    lambda: mxmoe.fp8_block128_grouped_gemm(u8(4, 256), f32(4, 2), u8(3, 8, 256), f32(3, 1, 2), i32(3), bf(4, 8)),
    lambda: mxmoe.fp8_block128_grouped_gemm(u8(4, 256), f32(4, 2), u8(3, 8, 256), f32(3, 2, 2), i32(4), bf(4, 8)),
    lambda: mxmoe.fp8_block128_grouped_gemm(u8(4, 256), f32(4, 2), u8(3, 8, 256), f32(3, 1, 2), i32(4).long(), bf(4, 8)),
    lambda: mxmoe.fp8_block128_grouped_wgrad(u8(8, 256), f32(8, 2), u8(16, 256), f32(16, 2), i32(4), f32(8, 16)),
    lambda: mxmoe.fp8_block128_grouped_wgrad(u8(8, 250), f32(8, 1), u8(16, 250), f32(16, 1), i32(4), f32(3, 8, 16)),
    lambda: mxmoe.fp8_block128_grouped_wgrad(u8(8, 256), f32(8, 2), u8(16, 128), f32(16, 2), i32(4), f32(3, 8, 16)),
    lambda: mxmoe.fp8_block128_grouped_wgrad(u8(8, 256), f32(8, 2), u8(16, 256), f32(16, 1), i32(4), f32(3, 8, 16)),
])
def test_binding_refuses_wrong_tensors(monkeypatch, lib, call):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(mxmoe, "_torch", None)
    with pytest.raises(ValueError):
        call()
    mxmoe._torch = None
