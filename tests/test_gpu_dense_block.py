"""The dense block in microscaled formats on the GPU: mx_add_rmsnorm,
mx_swiglu_quantize, mx_dequantize, fp4_block_gemm and fp4_dense_ffn against
their plain 64-bit forms, at the sizes where each can go wrong.

Tolerances.  Codes, scales, h and n are compared bit for bit: h is fp32
additions in a fixed order, and n and the SwiGLU are evaluated in double and
rounded once, so they can differ from the 64-bit form only where two doubles
a few 2^-53 apart straddle an fp32 rounding border.  Products of E2M1 by E2M1
are multiples of a common power of two per pair of scales; the accumulator
takes K in pieces of 64, so with S = ceil(K / 64) roundings (or truncations)
of fp32 each partial sum, at most A = sum |a w|, is off by at most S 2^-23 A.
For E4M3 activations the matrix cores round inside a piece; those results are
held to the library's bar for fp32-accumulated outputs (2e-3 of the largest,
cosine 0.99999).  A bf16 result is the fp32 one rounded: 2^-8 relative more,
and bit for bit the rounding of the fp32 call's result."""
import numpy as np
import pytest
import torch

import dense_block_ref as ref
from block_scaled_fp8xfp4_amd import mxmoe
from block_scaled_fp8xfp4_amd.layer import AddNorm, DenseFFN, FP4Linear
from dense_block_ref import E2M1, E4M3, codes_like, to_dev
from gpu_common import assert_close, host, say

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def typed(v, dtype):
    """(device tensor of dtype, its fp32 values) of fp32 values."""
    t = torch.from_numpy(np.ascontiguousarray(v, np.float32)).to(dtype)
    return t.cuda(), t.float().numpy()


def same_bits(got, want, what):
    g, w = host(got), np.ascontiguousarray(want)
    bad = np.flatnonzero(g.reshape(-1).view(np.uint8) != w.reshape(-1).view(np.uint8))
    assert bad.size == 0, f"{what}: {bad.size} bytes differ, first at {bad[:4]}"


# ------------------------------------------------------------------ norm
NORM_CASES = [  # T, H, x, residual, addends, weight, fmt
    (1, 4096, F32, BF16, 2, BF16, E4M3), (1, 32, BF16, None, 1, None, E2M1), (3, 64, F32, None, 2, F32, E4M3),
    (5, 2016, BF16, F32, 1, BF16, E2M1), (7, 2048, F32, F32, 2, F32, E2M1), (33, 2080, BF16, BF16, 1, BF16, E4M3),
    (2, 4128, F32, BF16, 1, None, E4M3), (48, 5120, BF16, BF16, 2, F32, E2M1), (4, 8192, BF16, BF16, 1, BF16, E4M3),
    (3, 8224, F32, BF16, 1, BF16, E2M1), (2, 16384, BF16, F32, 2, BF16, E4M3), (257, 992, BF16, BF16, 1, BF16, E4M3),
]


@pytest.mark.parametrize("T,H,xt,rt,addends,wt,fmt", NORM_CASES)
def test_add_rmsnorm(T, H, xt, rt, addends, wt, fmt):
    rng = np.random.default_rng(T * 31 + H)
    x, xv = typed(ref.activations(rng, T, H), xt)
    x2, x2v = typed(ref.activations(rng, T, H), xt) if addends == 2 else (None, None)
    r, rv = typed(ref.activations(rng, T, H) * 3, rt) if rt is not None else (None, None)
    w, wv = typed(1 + 0.1 * rng.standard_normal(H), wt) if wt is not None else (None, None)
    q, sc = codes_like(T, H, fmt)
    n = torch.empty((T, H), dtype=BF16, device="cuda")
    h = torch.empty_like(r) if r is not None else None
    mxmoe.mx_add_rmsnorm(x, w, 1e-6, residual=r, x2=x2, h=h, n=n, q=q, sc=sc, fmt=fmt)
    rh, rn = ref.add_rmsnorm(xv, rv, x2v, wv, 1e-6, rt == BF16)
    rq, rs = ref.quantize(rn, fmt)
    if h is not None:
        same_bits(h.float(), rh, "h")
    same_bits(n.float(), ref.bf16(rn), "n")
    same_bits(sc, rs, "scales")
    same_bits(q, rq, "codes")


def test_add_rmsnorm_rows_do_not_depend_on_T_and_outputs_are_optional():
    T, H = 70, 1056
    rng = np.random.default_rng(2)
    x, _ = typed(ref.activations(rng, T, H), BF16)
    r, _ = typed(ref.activations(rng, T, H), BF16)
    w, _ = typed(1 + 0.1 * rng.standard_normal(H), BF16)
    q, sc = codes_like(T, H, E4M3)
    h, n = torch.empty_like(r), torch.empty_like(r)
    mxmoe.mx_add_rmsnorm(x, w, 1e-5, residual=r, h=h, n=n, q=q, sc=sc)
    for t0, t1 in ((0, 1), (17, 19), (3, 70)):
        q1, s1 = codes_like(t1 - t0, H, E4M3)
        mxmoe.mx_add_rmsnorm(x[t0:t1], w, 1e-5, residual=r[t0:t1], q=q1, sc=s1)          # neither h nor n
        assert torch.equal(q1, q[t0:t1]) and torch.equal(s1, sc[t0:t1])
    n2 = torch.empty_like(n)
    mxmoe.mx_add_rmsnorm(h, w, 1e-5, n=n2)                                                # the norm of what was stored
    assert torch.equal(n2, n)
    h2 = torch.empty_like(h)
    mxmoe.mx_add_rmsnorm(x, None, 1e-5, residual=r, h=h2)                                 # the addition alone
    assert torch.equal(h2, h)
    r2 = r.clone()
    mxmoe.mx_add_rmsnorm(x, w, 1e-5, residual=r2, h=r2, n=n2)                             # in place
    assert torch.equal(r2, h) and torch.equal(n2, n)
    h3 = torch.empty((T, H), dtype=BF16, device="cuda")
    mxmoe.mx_add_rmsnorm(x.float(), w, 1e-5, h=h3, n=n2)                                  # h without a residual: x rounded
    assert torch.equal(h3, x)


def test_add_rmsnorm_strides_zero_rows_and_untouched_memory():
    """Rows inside wider buffers, a row of zeros, huge and tiny rows; nothing outside the rows is written."""
    T, H, pad = 6, 160, 24
    rng = np.random.default_rng(5)
    v = ref.activations(rng, T, H)
    v[2] = 0.0
    v[3] *= 1e18
    v[4] *= 1e-18
    wide, _ = typed(np.pad(v, ((0, 0), (8, pad - 8))), F32)
    res = torch.zeros((T, H + pad), dtype=F32, device="cuda")
    hw = torch.full((T + 1, H + pad), 7.0, dtype=F32, device="cuda")
    q, sc = codes_like(T + 1, H, E2M1)
    n = torch.full((T + 1, H), 7.0, dtype=BF16, device="cuda")
    mxmoe.mx_add_rmsnorm(wide[:, 8:8 + H], None, 1e-6, residual=res[:, :H], h=hw[:T, 8:8 + H], n=n[:T], q=q[:T],
                         sc=sc[:T], fmt=E2M1)
    rh, rn = ref.add_rmsnorm(v, np.zeros_like(v), None, None, 1e-6, False)
    rq, rs = ref.quantize(rn, E2M1)
    same_bits(hw[:T, 8:8 + H].contiguous(), rh, "h")
    same_bits(n[:T].float(), ref.bf16(rn), "n")
    same_bits(q[:T], rq, "codes")
    same_bits(sc[:T], rs, "scales")
    assert np.all(rn[2] == 0) and np.isfinite(rn).all()
    assert torch.all(hw[:, :8] == 7) and torch.all(hw[:, 8 + H:] == 7) and torch.all(hw[T] == 7)
    assert torch.all(n[T] == 7) and torch.all(q[T] == 0xA5) and torch.all(sc[T] == 0xA5)


# --------------------------------------------------------- SwiGLU + codes
@pytest.mark.parametrize("fmt", [E4M3, E2M1])
@pytest.mark.parametrize("T,I,dtype,pad", [(1, 32, F32, 0), (1, 576, BF16, 0), (3, 1376, F32, 8), (130, 96, BF16, 16),
                                           (9, 2048, BF16, 0), (2, 16384, F32, 0)])
def test_swiglu_quantize(T, I, dtype, pad, fmt):
    rng = np.random.default_rng(T + I)
    gu = ref.activations(rng, T, 2 * I) * 2
    gu[0, :8] = [0.0, -0.0, 1e-30, -1e-30, 88.0, -88.0, 200.0, -750.0]
    gu[-1, I:I + 32] = 0.0
    t, v = typed(np.pad(gu, ((0, 0), (0, pad))), dtype)
    q, sc = codes_like(T + 1, I, fmt)
    mxmoe.mx_swiglu_quantize(t[:, :2 * I], q[:T], sc[:T], fmt)
    rq, rs = ref.quantize(ref.swiglu(v[:, :2 * I]), fmt)
    same_bits(sc[:T], rs, "scales")
    same_bits(q[:T], rq, "codes")
    assert torch.all(q[T] == 0xA5) and torch.all(sc[T] == 0xA5)


def test_swiglu_quantize_on_rounding_borders():
    """Values placed on the borders between codes, and next to them: gate large (silu(g) = g in fp32's
    precision), up at the midpoints of each format times powers of two and one fp32 step beside them."""
    for fmt, grid in ((E4M3, [1 + m / 8 + 1 / 16 for m in range(8)] + [2.0 ** -10, 3 * 2.0 ** -10]),
                      (E2M1, [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])):
        mids = np.array(grid, np.float32)
        mids = np.concatenate([np.nextafter(mids, np.float32(0)), mids, np.nextafter(mids, np.float32(1e9))])
        up = np.zeros((1, 64), np.float32)
        top = 448.0 if fmt == E4M3 else 6.0
        up[0, 0], up[0, 32] = top, -top                                   # the block's largest fixes the scale
        k = min(31, mids.size)
        up[0, 1:1 + k], up[0, 33:33 + k] = mids[:k], -mids[-k:]
        gate = np.full((1, 64), 64.0, np.float32)
        gu = np.concatenate([gate, up / 64.0], -1)
        q, sc = codes_like(1, 64, fmt)
        mxmoe.mx_swiglu_quantize(to_dev(gu), q, sc, fmt)
        rq, rs = ref.quantize(ref.swiglu(gu), fmt)
        same_bits(sc, rs, "scales")
        same_bits(q, rq, "codes")


# ------------------------------------------------------------- dequantize
@pytest.mark.parametrize("fmt", [E4M3, E2M1])
def test_dequantize_every_code_and_scale(fmt):
    """Every element code under every scale: fp32 is the exact value (or infinity past its range), bf16 its rounding."""
    per = 256 if fmt == E4M3 else 16
    codes = np.arange(256, dtype=np.uint8)
    if fmt == E4M3:
        codes = np.where((codes & 127) == 127, 0, codes)
        q = np.repeat(codes[None], 255, 0)
    else:
        q = np.repeat(codes[None], 255, 0)
    cols = q.shape[1] * (1 if fmt == E4M3 else 2)
    sc = np.repeat(np.arange(255, dtype=np.uint8)[:, None], cols // 32, 1)
    want = ref.values(q, sc, fmt)
    with np.errstate(over="ignore"):
        want32 = want.astype(np.float32)
    for dtype in (F32, BF16):
        out = torch.empty((255, cols), dtype=dtype, device="cuda")
        mxmoe.mx_dequantize(to_dev(q), to_dev(sc), fmt, out)
        same_bits(out.float(), want32 if dtype == F32 else ref.bf16(want32), f"{per} codes")
    if fmt == E4M3:
        out = torch.empty((1, 32), dtype=F32, device="cuda")
        mxmoe.mx_dequantize(torch.full((1, 32), 0xFF, dtype=torch.uint8, device="cuda"),
                            torch.full((1, 1), 127, dtype=torch.uint8, device="cuda"), fmt, out)
        assert torch.isnan(out).all()


@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 1056), (257, 4096)])
@pytest.mark.parametrize("fmt", [E4M3, E2M1])
def test_dequantize_inverts_quantize(rows, cols, fmt):
    rng = np.random.default_rng(rows)
    v = ref.activations(rng, rows, cols)
    q, sc = codes_like(rows, cols, fmt)
    mxmoe.mx_quantize(to_dev(v), q, sc, fmt)
    out = torch.full((rows + 1, cols), 7.0, dtype=BF16, device="cuda")
    mxmoe.mx_dequantize(q, sc, fmt, out[:rows])
    same_bits(out[:rows].float(), ref.values(*ref.quantize(v, fmt), fmt).astype(np.float32), "values")
    assert torch.all(out[rows] == 7)


# ---------------------------------------------------------------- product
def check_product(y32, y16, want, room, K, a_fmt):
    steps = -(-K // 64)
    got = host(y32).astype(np.float64)
    if a_fmt == E2M1:
        over = np.abs(got - want) - steps * 2.0 ** -23 * room
        assert over.max() <= 0, f"fp32 result off by {over.max():.3e} more than its bound"
    else:
        assert_close(got, want, "fp32 result")
    assert torch.equal(y16, y32.to(BF16)), "the bf16 result is the fp32 result rounded"


PRODUCT_SIZES = [(1, 1, 32), (1, 16, 128), (1, 4096, 4096), (2, 100, 96), (3, 17, 160), (15, 33, 544), (16, 64, 1024),
                 (17, 48, 576), (33, 1152, 256), (48, 4096, 4096), (64, 130, 2080), (65, 300, 1056), (127, 129, 288),
                 (128, 128, 512), (130, 260, 4128), (255, 255, 640), (300, 520, 992), (513, 384, 256), (1000, 272, 1120),
                 (2, 40, 16384), (129, 40, 16384), (16, 8200, 96), (8192, 16, 160),
                 (4100, 7, 544), (500, 250, 64)]


@pytest.mark.parametrize("a_fmt", [E4M3, E2M1])
@pytest.mark.parametrize("M,N,K", PRODUCT_SIZES)
def test_fp4_block_gemm(M, N, K, a_fmt):
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    a, a_sc = ref.quantize(ref.activations(rng, M, K), a_fmt)
    w, w_sc = ref.weights(rng, N, K)
    d = [to_dev(t) for t in (a, a_sc, w, w_sc)]
    y32 = torch.full((M + 1, N), float("nan"), dtype=F32, device="cuda")
    y16 = torch.full((M + 1, N), float("nan"), dtype=BF16, device="cuda")
    mxmoe.fp4_block_gemm(d[0], d[1], a_fmt, d[2], d[3], y32[:M])
    v = mxmoe.last_variant()
    mxmoe.fp4_block_gemm(d[0], d[1], a_fmt, d[2], d[3], y16[:M])
    check_product(y32[:M], y16[:M], *ref.product(a, a_sc, a_fmt, w, w_sc), K, a_fmt)
    assert torch.isnan(y32[M]).all() and torch.isnan(y16[M]).all()
    say(f"{v}: {M} x {N} x {K}")


@pytest.mark.parametrize("a_fmt", [E4M3, E2M1])
def test_fp4_block_gemm_wide_scales(a_fmt):
    """Blocks whose scales lie far apart (partial sums that do not fit 24 bits), the scales' ends 0 and 254, zeros."""
    M, N, K = 40, 72, 1024
    rng = np.random.default_rng(9)
    codes = rng.integers(0, 256, (M, K if a_fmt == E4M3 else K // 2), dtype=np.uint8)
    if a_fmt == E4M3:
        codes = np.where((codes & 0x78) == 0x78, codes & 0x87, codes)     # no NaN, exponents below the top
    w = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    a_sc = rng.integers(115, 140, (M, K // 32)).astype(np.uint8)
    w_sc = rng.integers(115, 140, (N, K // 32)).astype(np.uint8)
    a_sc[0], w_sc[0] = 0, 127                                             # 2^-127: subnormal products
    a_sc[1] = 254
    codes[2] = 0
    d = [to_dev(t) for t in (codes, a_sc, w, w_sc)]
    y32 = torch.empty((M, N), dtype=F32, device="cuda")
    mxmoe.fp4_block_gemm(d[0], d[1], a_fmt, d[2], d[3], y32)
    want, room = ref.product(codes, a_sc, a_fmt, w, w_sc)
    got = host(y32).astype(np.float64)
    assert np.all(got[2] == 0)
    big = np.abs(want) < 2.0 ** 126
    rows = slice(3, M)
    steps = K // 64
    bound = (steps * 2.0 ** -23 if a_fmt == E2M1 else 2e-3) * room
    assert np.all((np.abs(got - want) <= bound)[rows])
    assert np.all(np.abs(got[0] - want[0]) <= bound[0] + 2.0 ** -126)     # results under the normal range may be flushed
    assert np.all((np.abs(got - want) <= bound)[1][big[1]])


@pytest.mark.parametrize("a_fmt", [E4M3, E2M1])
@pytest.mark.parametrize("N,K", [(4096, 4096), (520, 992), (96, 2080)])
def test_fp4_block_gemm_rows_do_not_depend_on_M(N, K, a_fmt):
    """The same row alone, in every batch size around the kernels' borders and inside a large batch: same bits."""
    rng = np.random.default_rng(N + K)
    M = 600
    a, a_sc = ref.quantize(ref.activations(rng, M, K), a_fmt)
    w, w_sc = ref.weights(rng, N, K)
    a, a_sc, w, w_sc = (to_dev(t) for t in (a, a_sc, w, w_sc))
    whole = torch.empty((M, N), dtype=F32, device="cuda")
    mxmoe.fp4_block_gemm(a, a_sc, a_fmt, w, w_sc, whole)
    seen = {mxmoe.last_variant()}
    for m in (1, 2, 5, 16, 17, 31, 32, 33, 48, 63, 64, 65, 96, 127, 128, 129, 191, 192, 256, 257, 320, 511, 512):
        m0 = M - m if m % 2 else 0
        y = torch.empty((m, N), dtype=F32, device="cuda")
        mxmoe.fp4_block_gemm(a[m0:m0 + m], a_sc[m0:m0 + m], a_fmt, w, w_sc, y)
        seen.add(mxmoe.last_variant())
        assert torch.equal(y.view(torch.int32), whole[m0:m0 + m].view(torch.int32)), (m, mxmoe.last_variant())
    say(f"N {N} K {K}: rows equal over {sorted(seen)}")


def random_codes(rng, rows, K, fmt):
    """Any codes and scales near 1, no NaN: (codes, scales) in numpy."""
    q = rng.integers(0, 256, (rows, K if fmt == E4M3 else K // 2), dtype=np.uint8)
    if fmt == E4M3:
        q = np.where((q & 0x7F) == 0x7F, q & 0x87, q)
    return q, rng.integers(120, 134, (rows, K // 32)).astype(np.uint8)


@pytest.mark.parametrize("a_fmt", [E4M3, E2M1])
@pytest.mark.parametrize("whole", [0, 1, 2, 3, 4, 5, 7, 8, 9, 12, 15, 16, 17, 24])
def test_fp4_block_gemm_few_rows_at_every_end_of_K(whole, a_fmt):
    """K around the pieces of 512 and the number of them that few rows keep in flight; rows and columns that end early."""
    N = 40
    for tail in (0, 32, 96, 128, 224, 480):
        K = 512 * whole + tail
        if K == 0:
            continue
        rng = np.random.default_rng(K)
        a, a_sc = random_codes(rng, 16, K, a_fmt)
        w, w_sc = random_codes(rng, N, K, E2M1)
        want, room = ref.product(a, a_sc, a_fmt, w, w_sc)
        a, a_sc, w, w_sc = (to_dev(t) for t in (a, a_sc, w, w_sc))
        for M in (16, 1, 7, 9):
            y32 = torch.full((M + 1, N), float("nan"), dtype=F32, device="cuda")
            y16 = torch.full((M + 1, N), float("nan"), dtype=BF16, device="cuda")
            mxmoe.fp4_block_gemm(a[16 - M:], a_sc[16 - M:], a_fmt, w, w_sc, y32[:M])
            mxmoe.fp4_block_gemm(a[16 - M:], a_sc[16 - M:], a_fmt, w, w_sc, y16[:M])
            check_product(y32[:M], y16[:M], want[16 - M:], room[16 - M:], K, a_fmt)
            assert torch.isnan(y32[M]).all() and torch.isnan(y16[M]).all(), (K, M)


@pytest.mark.parametrize("a_fmt", [E4M3, E2M1])
@pytest.mark.parametrize("M,N", [(40, 2801), (1040, 523), (1500, 1502), (2100, 2835), (2830, 2835)])
def test_fp4_block_gemm_tiles_at_every_end_of_K(M, N, a_fmt):
    """K around the stages and the K = 512 of scales of each tile: the bits of few rows, at the first, a middle and the last
    rows, columns that end inside a tile at odd addresses, and nothing written behind."""
    for K in (128, 160, 192, 256, 288, 384, 512, 544, 608, 640, 768, 896, 1024, 1056, 1280, 1536, 1632, 2048, 2080, 4096):
        rng = np.random.default_rng(K + M)
        a, a_sc, w, w_sc = (to_dev(t) for t in random_codes(rng, M, K, a_fmt) + random_codes(rng, N, K, E2M1))
        for dtype in (F32, BF16):
            off = 1 if dtype == F32 else 2                # four bytes: what y has to be aligned to
            buf = torch.full((M * N + 64,), float("nan"), dtype=dtype, device="cuda")
            y = buf[off:off + M * N].view(M, N)
            mxmoe.fp4_block_gemm(a, a_sc, a_fmt, w, w_sc, y)
            v = mxmoe.last_variant()
            assert "tile" in v
            for m0 in (0, M // 2 - 3, M - 16):
                few = torch.empty((16, N), dtype=dtype, device="cuda")
                mxmoe.fp4_block_gemm(a[m0:m0 + 16], a_sc[m0:m0 + 16], a_fmt, w, w_sc, few)
                if 16 * K * (2 if a_fmt == E4M3 else 1) < 2 ** 17:
                    assert "tile" not in mxmoe.last_variant()
                assert torch.equal(y[m0:m0 + 16], few), (K, m0, dtype, v)
            assert not torch.isnan(y).any(), (K, dtype, v)
            assert torch.isnan(buf[:off]).all() and torch.isnan(buf[off + M * N:]).all(), (K, dtype, v)
    say(f"{v}: {M} x {N}")


# -------------------------------------------------------------- dense FFN
FFN_SIZES = [(1, 4096, 576), (1, 256, 64), (1, 128, 2048), (2, 32, 32), (3, 160, 96), (16, 512, 256), (17, 1056, 544),
             (48, 4096, 576), (100, 288, 1376), (129, 512, 160), (300, 640, 736), (600, 256, 512), (1, 16384, 32),
             (5, 96, 16384), (7, 4096, 576), (2, 4096, 2048), (16, 4096, 160), (4, 8224, 2016)]


@pytest.mark.parametrize("x_fmt,mid_fmt", [(E4M3, E4M3), (E2M1, E2M1), (E4M3, E2M1), (E2M1, E4M3)])
@pytest.mark.parametrize("T,H,I", FFN_SIZES)
def test_fp4_dense_ffn_is_its_three_steps(T, H, I, x_fmt, mid_fmt):
    rng = np.random.default_rng(T + H + I)
    x, x_sc = (to_dev(t) for t in ref.quantize(ref.activations(rng, T, H), x_fmt))
    w13, w13_sc, w2, w2_sc = (to_dev(t) for t in ref.weights(rng, 2 * I, H) + ref.weights(rng, H, I))
    gu = torch.empty((T, 2 * I), dtype=F32, device="cuda")
    mxmoe.fp4_block_gemm(x, x_sc, x_fmt, w13, w13_sc, gu)
    q, sc = codes_like(T, I, mid_fmt)
    mxmoe.mx_swiglu_quantize(gu, q, sc, mid_fmt)
    need = mxmoe.fp4_dense_ffn_workspace_bytes(T, H, I, mid_fmt)
    for dtype in (F32, BF16):
        want = torch.empty((T, H), dtype=dtype, device="cuda")
        mxmoe.fp4_block_gemm(q, sc, mid_fmt, w2, w2_sc, want)
        ws = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device="cuda")
        y = torch.full((T + 1, H), float("nan"), dtype=dtype, device="cuda")
        mxmoe.fp4_dense_ffn(x, x_sc, x_fmt, w13, w13_sc, w2, w2_sc, mid_fmt, y[:T], ws[:need])
        assert torch.equal(y[:T], want), mxmoe.last_variant()
        assert torch.isnan(y[T]).all() and torch.all(ws[need:] == 0xA5)
    say(f"{mxmoe.last_variant()}: T {T} H {H} I {I}")


@pytest.mark.parametrize("fmt", [E4M3, E2M1])
@pytest.mark.parametrize("T,H,I", [(5, 256, 96), (40, 256, 96), (40, 128, 4128), (600, 128, 1056), (1100, 160, 2080), (1500, 128, 2080), (2040, 544, 4064), (2100, 256, 4128),
                                   (8, 2048, 256), (16, 4096, 96), (3, 6240, 2080)])
def test_fp4_dense_ffn_blocks_that_need_double(T, H, I, fmt):
    """Gates far below zero and products next to fp32's ends, whose codes fp32 does not decide, zero rows and gates whose
    SwiGLU vanishes, in every kernel of the gate/up product: the codes of mx_swiglu_quantize on the product's own result."""
    rng = np.random.default_rng(T + I)
    x, x_sc = random_codes(rng, T, H, fmt)
    w13, w13_sc = random_codes(rng, 2 * I, H, E2M1)
    w2, w2_sc = random_codes(rng, H, I, E2M1)
    x[T // 3] = 0                                                         # a row of zeros
    x_sc[T // 2] = 141                                                    # gates in the thousands, both signs
    x_sc[T - 1] = 20                                                      # subnormal blocks
    w13_sc[3] = 100
    x, x_sc, w13, w13_sc, w2, w2_sc = (to_dev(t) for t in (x, x_sc, w13, w13_sc, w2, w2_sc))
    gu = torch.empty((T, 2 * I), dtype=F32, device="cuda")
    mxmoe.fp4_block_gemm(x, x_sc, fmt, w13, w13_sc, gu)
    assert float(gu[:, :I].min()) < -1000
    q, sc = codes_like(T, I, fmt)
    mxmoe.mx_swiglu_quantize(gu, q, sc, fmt)
    want = torch.empty((T, H), dtype=F32, device="cuda")
    mxmoe.fp4_block_gemm(q, sc, fmt, w2, w2_sc, want)
    ws = torch.empty(mxmoe.fp4_dense_ffn_workspace_bytes(T, H, I, fmt), dtype=torch.uint8, device="cuda")
    y = torch.empty((T, H), dtype=F32, device="cuda")
    mxmoe.fp4_dense_ffn(x, x_sc, fmt, w13, w13_sc, w2, w2_sc, fmt, y, ws)
    assert torch.equal(y.view(torch.int32), want.view(torch.int32)), mxmoe.last_variant()
    say(f"{mxmoe.last_variant()}: T {T} H {H} I {I}")


def test_fp4_dense_ffn_rows_do_not_depend_on_T():
    rng = np.random.default_rng(11)
    T, H, I = 530, 512, 544
    x, x_sc = (to_dev(t) for t in ref.quantize(ref.activations(rng, T, H), E4M3))
    w13, w13_sc, w2, w2_sc = (to_dev(t) for t in ref.weights(rng, 2 * I, H) + ref.weights(rng, H, I))
    ffn = DenseFFN(w13, w13_sc, w2, w2_sc, T)
    whole = ffn(x, x_sc, E4M3, dtype=F32)
    for t in (1, 2, 15, 33, 64, 65, 128, 200, 257):
        assert torch.equal(ffn(x[-t:], x_sc[-t:], E4M3, dtype=F32), whole[-t:]), t


# ------------------------------------------------- together, as they are used
@pytest.mark.parametrize("T", [1, 6, 200])
def test_dense_block_runs_together(T):
    """Two layers of a model: norm -> FP4 projection; residual -> norm -> dense FFN; its output and a second addend ->
    residual -> norm in bf16 for the router logits.  Each step against the 64-bit form of the step's own inputs."""
    H, I, E = 512, 288, 24
    rng = np.random.default_rng(T)
    res, rv = typed(ref.activations(rng, T, H), BF16)
    x, xv = typed(ref.activations(rng, T, H), BF16)
    w, wv = typed(1 + 0.1 * rng.standard_normal(H), BF16)
    wp = [to_dev(t) for t in ref.weights(rng, H, H)]
    wf = [to_dev(t) for t in ref.weights(rng, 2 * I, H) + ref.weights(rng, H, I)]
    norm, proj, ffn = AddNorm(w, 1e-6), FP4Linear(*wp), DenseFFN(*wf, T, mid_fmt=E2M1)

    h, q, sc = norm(x, res, fmt=E4M3)
    rh, rn = ref.add_rmsnorm(xv, rv, None, wv, 1e-6, True)
    same_bits(h.float(), rh, "h")
    same_bits(q, ref.quantize(rn, E4M3)[0], "codes")
    y = proj(q, sc, E4M3)                                                  # bf16
    want = ref.product(host(q), host(sc), E4M3, host(wp[0]), host(wp[1]))[0]
    # the bar of the fp32 result, and its rounding to bf16: half a step, at most 2^-8 of the value
    assert np.all(np.abs(host(y.float()) - want) <= 2e-3 * np.abs(want).max() + 2.0 ** -8 * np.abs(want) * (1 + 2e-3))

    h2, q2, sc2 = norm(y, h, fmt=E2M1)
    rh2, rn2 = ref.add_rmsnorm(host(y.float()), rh, None, wv, 1e-6, True)
    same_bits(h2.float(), rh2, "h2")
    same_bits(q2, ref.quantize(rn2, E2M1)[0], "codes 2")
    f = ffn(q2, sc2, E2M1, dtype=F32)
    gu = ref.product(host(q2), host(sc2), E2M1, host(wf[0]), host(wf[1]))[0].astype(np.float32)
    mid = ref.quantize(ref.swiglu(gu), E2M1)
    want, room = ref.product(*mid, E2M1, host(wf[2]), host(wf[3]))
    # E2M1 sums are exact here (K 2^13 x 36 fits 24 bits under one scale; scales a few binades apart), so the
    # intermediate's codes are the reference's and the second product differs by its roundings at most
    assert np.all(np.abs(host(f) - want) <= -(-I // 64) * 2.0 ** -23 * room)

    x2, x2v = typed(ref.activations(rng, T, H), F32)
    h3, n3 = norm(f, h2, x2=x2, hidden=True)
    rh3, rn3 = ref.add_rmsnorm(host(f), rh2, x2v, wv, 1e-6, True)
    same_bits(h3.float(), rh3, "h3")
    same_bits(n3.float(), ref.bf16(rn3), "n3")
    gate = torch.from_numpy(rng.standard_normal((E, H)).astype(np.float32)).to(BF16).cuda()
    lg = torch.empty((T, E), dtype=F32, device="cuda")
    ws = torch.empty(max(256, mxmoe.moe_router_logits_workspace_bytes(T, H, E)), dtype=torch.uint8, device="cuda")
    mxmoe.moe_router_logits(n3, gate, lg, ws)
    assert_close(host(lg), host(n3.float()).astype(np.float64) @ host(gate.float()).astype(np.float64).T, "router logits")


@pytest.mark.parametrize("T", [1, 40, 300])
def test_dense_block_in_a_graph_and_on_another_stream(T):
    """The block captured once and replayed on new rows, between eager calls on the same stream and workspace; every
    replay against the eager result.  And the block on a side stream."""
    H, I = 512, 576
    rng = np.random.default_rng(T + 3)
    w = to_dev((1 + 0.1 * rng.standard_normal(H)).astype(np.float32))
    wf = [to_dev(t) for t in ref.weights(rng, 2 * I, H) + ref.weights(rng, H, I)]
    rows = [typed(ref.activations(rng, T, H), BF16)[0] for _ in range(4)]
    x, r = rows[0].clone(), rows[1].clone()
    ws = torch.empty(mxmoe.fp4_dense_ffn_workspace_bytes(T, H, I, E4M3), dtype=torch.uint8, device="cuda")

    def block(x, r, out):
        h, q, sc, y = out
        mxmoe.mx_add_rmsnorm(x, w, 1e-6, residual=r, h=h, q=q, sc=sc, fmt=E4M3)
        mxmoe.fp4_dense_ffn(q, sc, E4M3, *wf, E4M3, y, ws)

    def buffers():
        return (torch.empty((T, H), dtype=BF16, device="cuda"), *codes_like(T, H, E4M3),
                torch.empty((T, H), dtype=F32, device="cuda"))

    want = []
    for k in range(4):
        out = buffers()
        block(rows[k], rows[(k + 1) % 4], out)
        want.append([t.clone() for t in out])
    side, out = torch.cuda.Stream(), buffers()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(x, r, out)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want[0]))
    graph, gout, eager = torch.cuda.CUDAGraph(), buffers(), buffers()
    with torch.cuda.graph(graph):
        block(x, r, gout)
    for k in (1, 2, 3, 0, 2):
        x.copy_(rows[k])
        r.copy_(rows[(k + 1) % 4])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(gout, want[k])), k
        block(rows[(k + 2) % 4], rows[(k + 3) % 4], eager)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, want[(k + 2) % 4])), k


@pytest.mark.parametrize("T", [4, 70])
def test_two_graphs_and_two_streams_at_once(T):
    """Two captured blocks with workspaces of their own, replayed on two streams at the same time, over and over, while
    eager calls run on the current stream; rows behind the last one stay as they were."""
    H, I, K = 1056, 576, 5
    rng = np.random.default_rng(T)
    w = to_dev((1 + 0.1 * rng.standard_normal(H)).astype(np.float32))
    wf = [to_dev(t) for t in ref.weights(rng, 2 * I, H) + ref.weights(rng, H, I)]
    need = mxmoe.fp4_dense_ffn_workspace_bytes(T, H, I, E2M1)

    class Block:
        def __init__(self):
            self.x, self.r = (typed(ref.activations(rng, T, H), BF16)[0] for _ in range(2))
            self.h = torch.full((T + 1, H), 7.0, dtype=BF16, device="cuda")
            self.q, self.sc = codes_like(T + 1, H, E4M3)
            self.q.fill_(77)
            self.sc.fill_(77)
            self.y = torch.full((T + 1, H), 7.0, dtype=F32, device="cuda")
            self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")

        def run(self):
            mxmoe.mx_add_rmsnorm(self.x, w, 1e-6, residual=self.r, h=self.h[:T], q=self.q[:T], sc=self.sc[:T], fmt=E4M3)
            mxmoe.fp4_dense_ffn(self.q[:T], self.sc[:T], E4M3, *wf, E2M1, self.y[:T], self.ws)

    blocks = [Block() for _ in range(3)]
    want = []
    for b in blocks:
        b.run()
        want.append((b.h.clone(), b.q.clone(), b.y.clone()))
    graphs, streams = [torch.cuda.CUDAGraph() for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    for g, b in zip(graphs, blocks):
        with torch.cuda.graph(g):
            b.run()
    for b in blocks:
        b.h[:T].zero_()
        b.q[:T].zero_()
        b.y[:T].zero_()
    torch.cuda.synchronize()
    for k in range(K):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        blocks[2].run()
    torch.cuda.synchronize()
    for b, (h, q, y) in zip(blocks, want):
        assert torch.equal(b.h, h) and torch.equal(b.q, q) and torch.equal(b.y, y)
        assert torch.all(b.h[T] == 7) and torch.all(b.q[T] == 77) and torch.all(b.sc[T] == 77) and torch.all(b.y[T] == 7)


@pytest.mark.parametrize("a_fmt", [E4M3, E2M1])
@pytest.mark.parametrize("M,N,K", [(3, 48, 1056), (40, 2800, 1056), (300, 1040, 672), (1500, 1502, 1056), (2100, 2835, 1184),
                                   (2830, 2835, 1056)])
def test_fp4_block_gemm_scales_at_every_byte(M, N, K, a_fmt):
    """K % 128 != 0: scales that start at any byte, neighbours of other values around them."""
    rng = np.random.default_rng(M)
    a, a_sc, w, w_sc = random_codes(rng, M, K, a_fmt) + random_codes(rng, N, K, E2M1)
    da, dw = to_dev(a), to_dev(w)
    want = None
    for oa, ow in ((0, 0), (1, 3), (2, 2), (3, 1)):
        bufs = []
        for sc, o in ((a_sc, oa), (w_sc, ow)):
            b = torch.full((sc.size + 8,), 255, dtype=torch.uint8, device="cuda")
            b[o:o + sc.size] = to_dev(sc.reshape(-1))
            bufs.append(b[o:o + sc.size].view(sc.shape))
        y = torch.empty((M, N), dtype=F32, device="cuda")
        mxmoe.fp4_block_gemm(da, bufs[0], a_fmt, dw, bufs[1], y)
        assert not torch.isnan(y).any()
        want = y if want is None else want
        assert torch.equal(y, want), (oa, ow, mxmoe.last_variant())


def test_empty_batches():
    H, I = 64, 32
    e = lambda *s, dtype=torch.uint8: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    mxmoe.mx_add_rmsnorm(e(0, H, dtype=BF16), None, 1e-6, n=e(0, H, dtype=BF16))
    mxmoe.mx_swiglu_quantize(e(0, 2 * I, dtype=F32), e(0, I), e(0, 1), E4M3)
    mxmoe.mx_dequantize(e(0, H), e(0, 2), E4M3, e(0, H, dtype=F32))
    mxmoe.fp4_block_gemm(e(0, H), e(0, 2), E4M3, e(8, H // 2), e(8, 2), e(0, 8, dtype=F32))
    mxmoe.fp4_dense_ffn(e(0, H), e(0, 2), E4M3, e(2 * I, H // 2), e(2 * I, 2), e(H, I // 2), e(H, 1), E4M3,
                        e(0, H, dtype=F32), e(256))
    torch.cuda.synchronize()
