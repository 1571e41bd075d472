"""The dense block's entry points refuse bad arguments on the host, before
any HIP call: status codes of the C-ABI, ValueErrors of the binding."""
import ctypes
import os

import pytest
import torch

from block_scaled_fp8xfp4_amd import mxmoe
from block_scaled_fp8xfp4_amd.mxmoe import MX_EINVAL, MX_EUNSUPPORTED, MX_EWORKSPACE, MX_OK

FAKE = ctypes.c_void_p(1 << 20)        # aligned, never dereferenced: validation fails first
ODD = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mxmoe.LIB_PATH):
        import block_scaled_fp8xfp4_amd.build as b
        b.build()
    return mxmoe.load()


def norm(lib, x=FAKE, x2=None, xt=0, x_ld=64, r=FAKE, h=FAKE, rt=1, r_ld=64, w=FAKE, wt=1, T=4, H=64, eps=1e-6,
         n=FAKE, q=FAKE, sc=FAKE, fmt=0):
    return lib.mx_add_rmsnorm(x, x2, xt, x_ld, r, h, rt, r_ld, w, wt, T, H, eps, n, q, sc, fmt, None)


def test_add_rmsnorm_rejects_bad_arguments(lib):
    for bad in (dict(T=-1), dict(H=48), dict(H=0), dict(xt=2), dict(rt=5), dict(wt=-1), dict(fmt=2), dict(eps=0.0),
                dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")), dict(x_ld=32), dict(x_ld=66),
                dict(r_ld=60), dict(r_ld=68), dict(x=None), dict(sc=None), dict(q=None), dict(x=ODD), dict(x2=ODD),
                dict(r=ODD), dict(h=ODD), dict(w=ODD), dict(n=ODD), dict(q=ODD),
                dict(h=None, n=None, q=None, sc=None)):
        assert norm(lib, **bad) == MX_EINVAL, bad
    assert norm(lib, H=16416, x_ld=16416, r_ld=16416) == MX_EUNSUPPORTED
    assert norm(lib, x_ld=1 << 60) == MX_EUNSUPPORTED
    assert norm(lib, T=1 << 23) == MX_EUNSUPPORTED
    assert norm(lib, T=0, x=None, r=None, h=None, n=None, q=None, sc=None) == MX_OK


def test_swiglu_quantize_rejects_bad_arguments(lib):
    def call(gu=FAKE, dt=0, ld=128, T=4, I=64, fmt=0, q=FAKE, sc=FAKE):
        return lib.mx_swiglu_quantize(gu, dt, ld, T, I, fmt, q, sc, None)
    for bad in (dict(T=-1), dict(I=48), dict(I=0), dict(dt=2), dict(fmt=3), dict(ld=127), dict(ld=130),
                dict(dt=1, ld=132), dict(gu=None), dict(q=None), dict(sc=None), dict(gu=ODD), dict(q=ODD)):
        assert call(**bad) == MX_EINVAL, bad
    assert call(T=1 << 40, I=64) == MX_EUNSUPPORTED
    assert call(T=(1 << 28) + 1, I=64) == MX_EUNSUPPORTED          # 2^32 threads and more do not fit one launch
    assert call(T=0, gu=None, q=None, sc=None) == MX_OK


def test_dequantize_rejects_bad_arguments(lib):
    def call(q=FAKE, sc=FAKE, fmt=0, rows=4, cols=64, out=FAKE, dt=0):
        return lib.mx_dequantize(q, sc, fmt, rows, cols, out, dt, None)
    for bad in (dict(rows=-1), dict(cols=-32), dict(cols=40), dict(fmt=2), dict(dt=2), dict(q=None), dict(sc=None),
                dict(out=None), dict(q=ODD), dict(out=ODD)):
        assert call(**bad) == MX_EINVAL, bad
    assert call(rows=1 << 40) == MX_EUNSUPPORTED
    assert call(rows=(1 << 28) + 1) == MX_EUNSUPPORTED
    assert call(rows=0, q=None, sc=None, out=None) == MX_OK and call(cols=0) == MX_OK


def test_fp4_block_gemm_rejects_bad_arguments(lib):
    def call(a=FAKE, a_sc=FAKE, fmt=1, w=FAKE, w_sc=FAKE, M=4, N=5, K=128, y=FAKE, dt=0):
        return lib.fp4_block_gemm(a, a_sc, fmt, w, w_sc, M, N, K, y, dt, None)
    for bad in (dict(M=-1), dict(N=0), dict(K=0), dict(K=40), dict(fmt=2), dict(dt=2), dict(a=None), dict(a_sc=None),
                dict(w=None), dict(w_sc=None), dict(y=None), dict(a=ODD), dict(w=ODD), dict(a_sc=ODD), dict(w_sc=ODD),
                dict(y=ODD)):
        assert call(**bad) == MX_EINVAL, bad
    assert call(K=16416) == MX_EUNSUPPORTED
    assert call(M=1 << 20, N=1 << 20) == MX_EUNSUPPORTED
    assert call(M=1 << 28, N=1) == MX_EUNSUPPORTED and call(M=16, N=(1 << 30) - 63) == MX_EUNSUPPORTED
    assert call(M=0, a=None, a_sc=None, y=None) == MX_OK


def test_fp4_dense_ffn_rejects_bad_arguments(lib):
    big = 1 << 40

    def call(x=FAKE, x_sc=FAKE, xf=0, T=4, H=128, w13=FAKE, s13=FAKE, w2=FAKE, s2=FAKE, I=128, mf=0, y=FAKE, dt=0,
             ws=FAKE, n=big):
        return lib.fp4_dense_ffn(x, x_sc, xf, T, H, w13, s13, w2, s2, I, mf, y, dt, ws, n, None)
    for bad in (dict(T=-1), dict(H=40), dict(I=40), dict(I=0), dict(xf=2), dict(mf=2), dict(dt=2), dict(x=None),
                dict(x_sc=None), dict(w13=None), dict(s13=None), dict(w2=None), dict(s2=None), dict(y=None),
                dict(x=ODD), dict(x_sc=ODD), dict(w13=ODD), dict(w2=ODD), dict(s13=ODD), dict(s2=ODD), dict(y=ODD),
                dict(ws=ctypes.c_void_p((1 << 20) + 64))):
        assert call(**bad) == MX_EINVAL, bad
    assert call(H=16416) == MX_EUNSUPPORTED and call(I=16416) == MX_EUNSUPPORTED
    assert call(T=1 << 27, I=128) == MX_EUNSUPPORTED and call(T=1 << 27, H=256, I=32) == MX_EUNSUPPORTED
    assert call(ws=None) == MX_EWORKSPACE
    need = mxmoe.fp4_dense_ffn_workspace_bytes(4, 128, 128, 0)
    assert need > 0 and call(n=need - 1) == MX_EWORKSPACE
    assert call(T=0, x=None, x_sc=None, y=None, ws=None) == MX_OK
    for bad in ((-1, 64, 32, 0), (4, 40, 32, 0), (4, 64, 40, 0), (4, 64, 32, 2)):
        assert mxmoe.fp4_dense_ffn_workspace_bytes(*bad) == 0


def u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


def f32(*s):
    return torch.zeros(s, dtype=torch.float32)


def bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


@pytest.mark.parametrize("call", [
    lambda: mxmoe.mx_add_rmsnorm(f32(64), None, 1e-6, n=bf(1, 64)),
    lambda: mxmoe.mx_add_rmsnorm(f32(2, 64).half(), None, 1e-6, n=bf(2, 64)),
    lambda: mxmoe.mx_add_rmsnorm(f32(2, 64), None, 1e-6, n=f32(2, 64)),
    lambda: mxmoe.mx_add_rmsnorm(f32(2, 64), None, 1e-6, x2=bf(2, 64), n=bf(2, 64)),
    lambda: mxmoe.mx_add_rmsnorm(f32(2, 64), None, 1e-6, x2=f32(2, 128)[:, :64], n=bf(2, 64)),
    lambda: mxmoe.mx_add_rmsnorm(f32(2, 64), None, 1e-6, residual=bf(3, 64), n=bf(2, 64)),
    lambda: mxmoe.mx_add_rmsnorm(f32(2, 64), None, 1e-6, residual=bf(2, 64), h=f32(2, 64)),
    lambda: mxmoe.mx_add_rmsnorm(f32(2, 64), None, 1e-6, residual=bf(2, 64), h=bf(2, 128)[:, :64]),
    lambda: mxmoe.mx_add_rmsnorm(f32(64, 2).t(), None, 1e-6, n=bf(2, 64)),
    lambda: mxmoe.mx_add_rmsnorm(f32(2, 64)[:1].expand(2, 64), None, 1e-6, n=bf(2, 64)),
    lambda: mxmoe.mx_add_rmsnorm(f32(2, 64), f32(32), 1e-6, n=bf(2, 64)),
    lambda: mxmoe.mx_add_rmsnorm(f32(2, 64), None, 1e-6, q=u8(2, 64)),
    lambda: mxmoe.mx_add_rmsnorm(f32(2, 64), None, 1e-6, q=u8(2, 64), sc=u8(2, 2), fmt=mxmoe.MX_FMT_E2M1),
    lambda: mxmoe.mx_add_rmsnorm(f32(2, 64), None, 1e-6, q=u8(2, 64), sc=u8(2, 2), fmt=7),
    lambda: mxmoe.mx_swiglu_quantize(f32(2, 128), u8(2, 64), u8(2, 1), mxmoe.MX_FMT_E4M3),
    lambda: mxmoe.mx_swiglu_quantize(f32(2, 128), u8(2, 64), u8(2, 2), mxmoe.MX_FMT_E2M1),
    lambda: mxmoe.mx_swiglu_quantize(f32(128), u8(1, 64), u8(1, 2), mxmoe.MX_FMT_E4M3),
    lambda: mxmoe.mx_dequantize(u8(2, 64), u8(2, 2), mxmoe.MX_FMT_E4M3, f32(2, 128)),
    lambda: mxmoe.mx_dequantize(u8(2, 64), u8(2, 2), mxmoe.MX_FMT_E4M3, f32(2, 64).half()),
    lambda: mxmoe.mx_dequantize(u8(2, 128)[:, ::2], u8(2, 2), mxmoe.MX_FMT_E4M3, f32(2, 64)),
    lambda: mxmoe.fp4_block_gemm(u8(2, 64), u8(2, 2), mxmoe.MX_FMT_E2M1, u8(8, 32), u8(8, 2), f32(2, 8)),
    lambda: mxmoe.fp4_block_gemm(u8(2, 64), u8(2, 2), mxmoe.MX_FMT_E4M3, u8(8, 32), u8(8, 1), f32(2, 8)),
    lambda: mxmoe.fp4_block_gemm(u8(2, 64), u8(2, 2), mxmoe.MX_FMT_E4M3, u8(8, 32), u8(8, 2), f32(2, 9)),
    lambda: mxmoe.fp4_block_gemm(u8(2, 64), u8(2, 2), mxmoe.MX_FMT_E4M3, u8(8, 32), u8(8, 2), f32(8, 2).t()),
    lambda: mxmoe.fp4_dense_ffn(u8(2, 64), u8(2, 2), 0, u8(64, 32), u8(64, 2), u8(64, 32), u8(64, 1), 0, f32(2, 64), u8(9999)),
    lambda: mxmoe.fp4_dense_ffn(u8(2, 64), u8(2, 2), 0, u8(64, 32), u8(64, 2), u8(64, 16), u8(64, 1), 0, f32(3, 64), u8(9999)),
])
def test_binding_refuses_wrong_tensors(lib, call):
    with pytest.raises(ValueError):
        call()


def meta(*s, dtype=torch.uint8):
    return torch.empty(s, dtype=dtype, device="meta")


@pytest.mark.parametrize("call", [
    lambda n: mxmoe.mx_add_rmsnorm(meta(n, 32, dtype=torch.float32), None, 1e-6, n=meta(n, 32, dtype=torch.bfloat16)),
    lambda n: mxmoe.mx_add_rmsnorm(meta(1, n, dtype=torch.float32), None, 1e-6, n=meta(1, n, dtype=torch.bfloat16)),
    lambda n: mxmoe.mx_swiglu_quantize(meta(1, 2 * n, dtype=torch.float32), meta(1, n), meta(1, n // 32), mxmoe.MX_FMT_E4M3),
    lambda n: mxmoe.fp4_block_gemm(meta(n, 32), meta(n, 1), mxmoe.MX_FMT_E4M3, meta(8, 16), meta(8, 1),
                                   meta(n, 8, dtype=torch.float32)),
    lambda n: mxmoe.fp4_block_gemm(meta(2, n), meta(2, n // 32), mxmoe.MX_FMT_E4M3, meta(8, n // 2), meta(8, n // 32),
                                   meta(2, 8, dtype=torch.float32)),
    lambda n: mxmoe.fp4_block_gemm(meta(2, 32), meta(2, 1), mxmoe.MX_FMT_E4M3, meta(n, 16), meta(n, 1),
                                   meta(2, n, dtype=torch.float32)),
    lambda n: mxmoe.fp4_dense_ffn(meta(n, 32), meta(n, 1), 0, meta(64, 16), meta(64, 1), meta(32, 16), meta(32, 1), 0,
                                  meta(n, 32, dtype=torch.float32), meta(256)),
])
def test_binding_refuses_sizes_past_int(lib, call):
    """A size that does not fit the C-ABI's int would arrive cut: 2^32 + 32 as 32."""
    for n in (2**31, 2**32 + 32):
        with pytest.raises(ValueError, match="at most 2147483647"):
            call(n)
