"""Casts and products with a scale for each block of 128 against 64-bit forms.

Whole numbers under scales of few bits make every step of a product exact but its fp32 rounding, so the kernels' results are
compared bit for bit with the order of addition that they promise; other operands are compared within what the matrix cores
cut and fp32 rounds."""
import numpy as np
import pytest
import torch

import block128_ref as ref
from block128_ref import BF16, F32, U8, B, blocks, dev, typed
from block_scaled_fp8xfp4_amd import mxmoe

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1, 16), (1, 16, 128), (2, 130, 48), (3, 17, 144), (16, 300, 1040), (16, 64, 8208), (17, 100, 1040), (32, 48, 4112),
          (33, 65, 272), (64, 130, 2064), (65, 129, 384), (200, 333, 400), (130, 1030, 640), (1030, 260, 256), (600, 2050, 144)]


# ------------------------------------------------------------------- casts
def quantized(src, block_rows):
    q = torch.full(src.shape, 0xA5, dtype=U8, device="cuda")
    head = src.shape[:-2]
    sc = torch.full(head + (src.shape[-2] if block_rows == 1 else blocks(src.shape[-2]), blocks(src.shape[-1])), -1.0, device="cuda")
    mxmoe.fp8_quantize128(src, q, sc, block_rows)
    return q, sc


def loud(rng, rows, cols):
    return rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal(cols))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 128), (5, 144), (130, 400), (257, 1040)])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize(dtype, rows, cols, block_rows):
    src, v = typed(loud(np.random.default_rng(rows + cols), rows, cols), dtype)
    q, sc = quantized(src, block_rows)
    want_q, want_sc = ref.cast(v, block_rows, B)
    assert np.array_equal(sc.cpu().numpy(), want_sc) and np.array_equal(q.cpu().numpy(), want_q)


def test_quantize_matrices_and_rows_that_lie_apart():
    rng = np.random.default_rng(1)
    src, v = typed(loud(rng, 3 * 150, 208), BF16)
    q, sc = quantized(src.view(3, 150, 208), 128)
    for e in range(3):
        want_q, want_sc = ref.cast(v[e * 150:(e + 1) * 150], B, B)
        assert np.array_equal(sc[e].cpu().numpy(), want_sc) and np.array_equal(q[e].cpu().numpy(), want_q)
    for block_rows in (1, 128):
        part = src[:140, 16:176]
        q, sc = quantized(part, block_rows)
        want_q, want_sc = ref.cast(v[:140, 16:176], block_rows, B)
        assert np.array_equal(sc.cpu().numpy(), want_sc) and np.array_equal(q.cpu().numpy(), want_q)


def test_quantize_near_borders():
    """Quotients on and one fp32 step around every border between two codes, under scales of all mantissas; and blocks of
    zeros, of very small and of the largest numbers."""
    rng = np.random.default_rng(2)
    mids = (ref.E4M3_MAG[1:] + ref.E4M3_MAG[:-1]) / 2
    rows = []
    for i in range(200):
        amax = np.float32((1 + rng.random()) * 2.0 ** rng.integers(-50, 100))
        s = np.float64(np.float32(amax) / np.float32(448))
        x = (mids[rng.integers(0, len(mids), 127)] * s).astype(np.float32)
        x = np.where(rng.random(127) < 0.5, x, np.nextafter(x, np.float32(np.inf) * rng.choice([-1, 1], 127).astype(np.float32)))
        rows.append(np.concatenate([[amax], x * rng.choice([-1, 1], 127)]))
    for v in (0.0, 1e-45, 1e-30, 2.0**-60, 2.0**-59, 3.4028235e38):
        rows.append(np.full(128, v))
    src, v = typed(np.array(rows), F32)
    q, sc = quantized(src, 1)
    want_q, want_sc = ref.cast(v, 1, B)
    assert np.array_equal(sc.cpu().numpy(), want_sc) and np.array_equal(q.cpu().numpy(), want_q)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_quantize_infinities_and_nan(bad):
    """Their block's scale is NaN, other blocks are as without them."""
    src = torch.randn((200, 300), device="cuda")
    src = torch.nn.functional.pad(src, (0, 4))
    clean = [quantized(src, r) for r in (1, 128)]
    src[3, 130] = bad
    for (q0, s0), r in zip(clean, (1, 128)):
        q, sc = quantized(src, r)
        i = 3 if r == 1 else 0
        assert sc[i, 1].isnan() and sc.isnan().sum() == 1
        same = ~sc.isnan()
        assert torch.equal(sc[same], s0[same])
        keep = torch.ones_like(q, dtype=torch.bool)
        keep[i * r:(i + 1) * r, 128:256] = False
        assert torch.equal(q[keep], q0[keep])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,I", [(1, 16), (3, 144), (65, 576), (130, 1376)])
def test_swiglu_quantize(dtype, T, I):
    rng = np.random.default_rng(I)
    gu, v = typed(loud(rng, T, 2 * I) * 3, dtype)
    q, sc = torch.full((T, I), 0xA5, dtype=U8, device="cuda"), torch.full((T, blocks(I)), -1.0, device="cuda")
    mxmoe.fp8_swiglu_quantize128(gu, q, sc)
    g, u = v[:, :I], v[:, I:]
    a = (g / (1 + np.exp(-g)) * u).astype(np.float32)                 # double, rounded once
    # numpy's and the device's exponential may differ by the last bit of a double, which moves a rounding to fp32 once in
    # 2^28 elements: the few thousand here are compared exactly
    want_q, want_sc = ref.cast(a.astype(np.float64), 1, B)
    assert np.array_equal(sc.cpu().numpy(), want_sc) and np.array_equal(q.cpu().numpy(), want_q)
    wide = torch.zeros((T, 2 * I + 24), dtype=dtype, device="cuda")
    wide[:, 8:8 + 2 * I] = gu
    q2, sc2 = torch.zeros_like(q), torch.zeros_like(sc)
    mxmoe.fp8_swiglu_quantize128(wide[:, 8:8 + 2 * I], q2, sc2)
    assert torch.equal(q, q2) and torch.equal(sc, sc2)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_swiglu_quantize_many(dtype):
    """A million values, some next to a border between codes, and blocks whose largest value is there twice."""
    T, I = 1000, 1040
    gu, v = typed(np.random.default_rng(5).standard_normal((T, 2 * I)) * 4, dtype)
    for r in range(0, T, 50):
        top = int(np.abs(v[r, :128] / (1 + np.exp(-v[r, :128])) * v[r, I:I + 128]).argmax())
        for at in (0, I):
            v[r, at + (top + 1 + r // 50 * 7) % 128] = v[r, at + top]
    gu = torch.from_numpy(v).to(dtype).cuda()
    q, sc = torch.zeros((T, I), dtype=U8, device="cuda"), torch.zeros((T, blocks(I)), device="cuda")
    mxmoe.fp8_swiglu_quantize128(gu, q, sc)
    a = (v[:, :I] / (1 + np.exp(-v[:, :I])) * v[:, I:]).astype(np.float32)
    want_q, want_sc = ref.cast(a.astype(np.float64), 1, B)
    assert np.array_equal(sc.cpu().numpy(), want_sc) and np.array_equal(q.cpu().numpy(), want_q)


def test_swiglu_quantize_extremes():
    """Gates from far below to far above zero, subnormal ones, huge ones, and their ups; zero blocks."""
    g = np.concatenate([np.linspace(-110, 110, 97), [0, 1e-45, -1e-45, 1e-38, 3e38, -3e38, 88.8, -88.8, -745, -746],
                        np.random.default_rng(0).standard_normal(21)])
    gates = np.stack([np.roll(g, i) for i in range(128)])
    ups = np.stack([np.full(128, s) for s in np.float32(10.0) ** np.random.default_rng(1).integers(-30, 0, 128)])
    gu, v = typed(np.concatenate([gates, ups], 1), F32)
    q, sc = torch.zeros((128, 128), dtype=U8, device="cuda"), torch.zeros((128, 1), device="cuda")
    mxmoe.fp8_swiglu_quantize128(gu, q, sc)
    with np.errstate(over="ignore"):
        a = (v[:, :128] / (1 + np.exp(-v[:, :128])) * v[:, 128:]).astype(np.float32)
    want_q, want_sc = ref.cast(a.astype(np.float64), 1, B)
    assert np.array_equal(sc.cpu().numpy(), want_sc) and np.array_equal(q.cpu().numpy(), want_q)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bounds,cols,more", [([0, 1], 1, 0), ([0, 128], 64, 0), ([0, 300], 65, 0), ([0, 0, 5, 5, 133, 400, 400], 100, 0),
                                              ([0, 200, 330], 30, 50), (list(range(0, 300)), 7, 0), ([0, 0], 9, 4)])
def test_quantize_columns(dtype, bounds, cols, more):
    rows, E = bounds[-1] + more, len(bounds) - 1
    src, v = typed(loud(np.random.default_rng(cols), rows, cols), dtype)
    ld = mxmoe.fp8_quantize128_t_cols(rows, E)
    q, sc = torch.zeros((cols, ld), dtype=U8, device="cuda"), torch.zeros((cols, ld // B), device="cuda")
    mxmoe.fp8_quantize128_t(src, q, sc, dev(np.array(bounds, np.int32)))
    want_q, want_sc, _ = ref.columns(v, bounds, ld)
    assert np.array_equal(sc.cpu().numpy(), want_sc) and np.array_equal(q.cpu().numpy(), want_q)
    if E == 1 and not more:
        q2, sc2 = torch.zeros_like(q), torch.zeros_like(sc)
        mxmoe.fp8_quantize128_t(src, q2, sc2)
        assert torch.equal(q, q2) and torch.equal(sc, sc2)


# ---------------------------------------------------------------- products
def gemm(a, a_sc, w, w_sc, dtype):
    y = torch.full((a.shape[0], w.shape[0]), 7.0, dtype=dtype, device="cuda")
    mxmoe.fp8_block128_gemm(a, a_sc, w, w_sc, y)
    return y


@pytest.mark.parametrize("w_rows", [128, 1])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_in_order(M, N, K, w_rows):
    rng = np.random.default_rng(M + N + K)
    a, w = ref.whole_codes(rng, M, K), ref.whole_codes(rng, N, K)
    a_sc, w_sc = ref.short_scales(rng, M, blocks(K)), ref.short_scales(rng, -(-N // w_rows), blocks(K))
    want = ref.in_order(a, a_sc, w, w_sc, w_rows)
    args = [dev(v) for v in (a, a_sc, w, w_sc)]
    assert np.array_equal(gemm(*args, F32).cpu().numpy(), want)
    assert np.array_equal(gemm(*args, BF16).float().cpu().numpy(), ref.bf16(want))


@pytest.mark.parametrize("w_rows", [128, 1])
@pytest.mark.parametrize("M,N,K,variant", [(9, 4100, 400, "rows16"), (3, 9010, 272, "tile16x64"), (31, 4080, 272, "rows32"), (300, 1030, 656, "tile64x64"),
                                           (1030, 1100, 400, "tile64x128"), (2000, 1300, 272, "tile128x128"),
                                           (3001, 1500, 528, "tile128x256"), (6001, 1502, 400, "tile256x256"),
                                           (6000, 1500, 128, "tile256x256"), (6000, 1500, 16, "tile256x256")])
def test_every_kernel_in_order(M, N, K, variant, w_rows):
    rng = np.random.default_rng(M + N + K)
    a, w = ref.whole_codes(rng, M, K), ref.whole_codes(rng, N, K)
    a_sc, w_sc = ref.short_scales(rng, M, blocks(K)), ref.short_scales(rng, -(-N // w_rows), blocks(K))
    want = ref.in_order(a, a_sc, w, w_sc, w_rows)
    args = [dev(v) for v in (a, a_sc, w, w_sc)]
    assert np.array_equal(gemm(*args, F32).cpu().numpy(), want) and mxmoe.last_variant() == "b128:" + variant
    assert np.array_equal(gemm(*args, BF16).float().cpu().numpy(), ref.bf16(want))


@pytest.mark.parametrize("M", [1, 40, 300])
def test_product_long(M):
    rng = np.random.default_rng(M)
    N, K = 50, 33000 // 16 * 16
    a, w = ref.whole_codes(rng, M, K), ref.whole_codes(rng, N, K)
    a_sc, w_sc = ref.short_scales(rng, M, blocks(K)), ref.short_scales(rng, 1, blocks(K))
    got = gemm(*[dev(v) for v in (a, a_sc, w, w_sc)], F32)
    assert np.array_equal(got.cpu().numpy(), ref.in_order(a, a_sc, w, w_sc, 128))


@pytest.mark.parametrize("M,N,K", [(1, 512, 2048), (20, 300, 1040), (300, 700, 4096)])
def test_product_of_cast_values(M, N, K):
    """Against 64 bits.  The matrix cores cut each product at 2^-13 of the largest of its eight; a cut is at most that of the
    sum of magnitudes, 2^-13 * 8 of an eight's largest; fp32 rounds once per block, the scales' product once."""
    rng = np.random.default_rng(K)
    a, a_sc = ref.cast(loud(rng, M, K), 1, B)
    w, w_sc = ref.cast(rng.standard_normal((N, K)) * 0.02, B, B)
    av, wv = ref.wide(a, a_sc, 1), ref.wide(w, w_sc, B)
    want, most = av @ wv.T, np.abs(av) @ np.abs(wv).T
    got = gemm(*[dev(v) for v in (a, a_sc, w, w_sc)], F32).double().cpu().numpy()
    assert (np.abs(got - want) <= (2.0**-10 + (blocks(K) + 2) * 2.0**-23) * most).all()
    err = np.linalg.norm(got - want) / np.linalg.norm(want)
    print(f"{M} x {N} x {K}: {err:.2e} of the norm", flush=True)
    assert err <= 1e-4                # one product in ten cut, by 2^-14 of the largest on average: 2e-5 of the norm
    half = gemm(*[dev(v) for v in (a, a_sc, w, w_sc)], BF16)
    assert np.array_equal(half.float().cpu().numpy(), ref.bf16(got))


def test_a_row_does_not_depend_on_the_others():
    """The same bits alone, in few rows and in many: every kernel adds in the same order."""
    rng = np.random.default_rng(8)
    N, K = 1100, 1168
    a, a_sc = [dev(v) for v in ref.cast(loud(rng, 700, K), 1, B)]
    a, a_sc = a.repeat(25, 1), a_sc.repeat(25, 1)
    w, w_sc = [dev(v) for v in ref.cast(rng.standard_normal((N, K)), B, B)]
    variants, full = set(), gemm(a, a_sc, w, w_sc, F32)
    for M in (1, 2, 15, 16, 17, 31, 33, 48, 64, 65, 100, 129, 200, 257, 400, 700, 1200, 2500, 4000, 9000, 17000):
        y = gemm(a[-M:].contiguous(), a_sc[-M:].contiguous(), w, w_sc, F32)
        variants.add(mxmoe.last_variant())
        assert torch.equal(y, full[-M:]), M
    print(sorted(variants), flush=True)
    assert len(variants) == 7


def test_nan_scales_reach_their_rows_only():
    rng = np.random.default_rng(9)
    for M in (8, 400):
        a, a_sc, w, w_sc = [dev(v) for v in ref.cast(loud(rng, M, 256), 1, B) + ref.cast(loud(rng, 300, 256), B, B)]
        clean = gemm(a, a_sc, w, w_sc, F32)
        a_sc[5, 1] = float("nan")
        y = gemm(a, a_sc, w, w_sc, F32)
        assert y[5].isnan().all() and y.isnan().sum() == 300
        clean[5] = y[5] = 0
        assert torch.equal(y, clean)


def grouped(a, a_sc, w, w_sc, bounds, dtype):
    y = torch.full((a.shape[0], w.shape[1]), 7.0, dtype=dtype, device="cuda")
    mxmoe.fp8_block128_grouped_gemm(a, a_sc, w, w_sc, dev(np.array(bounds, np.int32)), y)
    return y


def ragged(rng, E, R):
    return [0] + sorted(int(v) for v in rng.integers(0, R + 1, E - 1)) + [R]


@pytest.mark.parametrize("E,R,more,N,K", [(1, 1, 0, 16, 128), (1, 300, 7, 130, 272), (3, 5, 2, 20, 48), (8, 8, 0, 200, 1040),
                                          (5, 70, 3, 65, 400), (16, 400, 9, 100, 256), (16, 3000, 100, 144, 272), (257, 1, 0, 33, 144),
                                          (257, 900, 5, 20, 144), (1024, 40, 0, 16, 16), (7, 0, 12, 40, 144), (4, 900, 0, 300, 656),
                                          (16, 1000, 30, 300, 400), (16, 300, 5, 520, 2064), (64, 1100, 0, 130, 528)])
def test_grouped_product_in_order(E, R, more, N, K):
    rng = np.random.default_rng(E + R)
    bounds = ragged(rng, E, R)
    a, a_sc = ref.whole_codes(rng, R + more, K), ref.short_scales(rng, R + more, blocks(K))
    w = ref.whole_codes(rng, E * N, K).reshape(E, N, K)
    w_sc = ref.short_scales(rng, E * blocks(N), blocks(K)).reshape(E, blocks(N), blocks(K))
    want = np.full((R + more, N), 7.0, np.float32)
    for e, (i, j) in enumerate(zip(bounds, bounds[1:])):
        if i < j:
            want[i:j] = ref.in_order(a[i:j], a_sc[i:j], w[e], w_sc[e], B)
    args = [dev(v) for v in (a, a_sc, w, w_sc)]
    assert np.array_equal(grouped(*args, bounds, F32).cpu().numpy(), want)
    print(mxmoe.last_variant(), flush=True)
    assert np.array_equal(grouped(*args, bounds, BF16).float().cpu().numpy(), ref.bf16(want))


def test_grouped_rows_equal_the_dense_product():
    rng = np.random.default_rng(11)
    E, N, K = 6, 200, 528
    a, a_sc = [dev(v) for v in ref.cast(loud(rng, 600, K), 1, B)]
    w, w_sc = zip(*[ref.cast(rng.standard_normal((N, K)), B, B) for _ in range(E)])
    w, w_sc = dev(np.stack(w)), dev(np.stack(w_sc))
    for bounds in ([0, 1, 1, 3, 20, 40, 600], [0, 2, 4, 6, 8, 10, 12]):
        R = bounds[-1]
        y = grouped(a[:R].contiguous(), a_sc[:R].contiguous(), w, w_sc, bounds, F32)
        for e, (i, j) in enumerate(zip(bounds, bounds[1:])):
            if i < j:
                assert torch.equal(y[i:j], gemm(a[i:j].contiguous(), a_sc[i:j].contiguous(), w[e], w_sc[e], F32))


def test_offsets_that_lie_stay_inside():
    """Offsets past the rows, below zero or descending: what they say is kept inside the rows that there are."""
    rng = np.random.default_rng(12)
    a, a_sc = ref.whole_codes(rng, 40, 144), ref.short_scales(rng, 40, 2)
    w, w_sc = ref.whole_codes(rng, 3 * 30, 144).reshape(3, 30, 144), ref.short_scales(rng, 3, 2).reshape(3, 1, 2)
    args = [dev(v) for v in (a, a_sc, w, w_sc)]
    want = np.full((40, 30), 7.0, np.float32)
    want[:25] = ref.in_order(a[:25], a_sc[:25], w[0], w_sc[0], B)
    want[25:] = ref.in_order(a[25:], a_sc[25:], w[1], w_sc[1], B)
    assert np.array_equal(grouped(*args, [-5, 25, 2**31 - 1, 90], F32).cpu().numpy(), want)
    src, v = typed(loud(rng, 40, 20), F32)
    q, sc = torch.zeros((20, 384), dtype=U8, device="cuda"), torch.zeros((20, 3), device="cuda")
    mxmoe.fp8_quantize128_t(src, q, sc, dev(np.array([-5, 25, 2**31 - 1, 90], np.int32)))
    want_q, want_sc, _ = ref.columns(v, [0, 25, 40], 384)
    assert np.array_equal(q.cpu().numpy(), want_q) and np.array_equal(sc.cpu().numpy(), want_sc)


@pytest.mark.parametrize("bounds,N,K", [([0, 1], 1, 1), ([0, 300], 130, 70), ([0, 0, 5, 5, 133, 400, 400], 100, 65),
                                        ([0, 1000, 1001], 33, 257), (list(range(0, 280)), 5, 7), ([0, 0, 0], 20, 30)])
def test_grouped_weight_gradient_in_order(bounds, N, K):
    rng = np.random.default_rng(N + K)
    E, rows = len(bounds) - 1, bounds[-1]
    ld = mxmoe.fp8_quantize128_t_cols(rows, E) + 128
    a, b = ref.whole_codes(rng, N, ld), ref.whole_codes(rng, K, ld)
    a_sc, b_sc = ref.short_scales(rng, N, ld // B), ref.short_scales(rng, K, ld // B)
    want, at = np.zeros((E, N, K), np.float32), 0
    for e, (i, j) in enumerate(zip(bounds, bounds[1:])):
        n = blocks(j - i)
        s, t = slice(at * B, (at + n) * B), slice(at, at + n)
        if n:
            want[e] = ref.in_order(a[:, s], a_sc[:, t], b[:, s], b_sc[:, t], 1)
        at += n
    for dtype in (F32, BF16):
        dw = torch.full((E, N, K), 7.0, dtype=dtype, device="cuda")
        mxmoe.fp8_block128_grouped_wgrad(*[dev(v) for v in (a, a_sc, b, b_sc)], dev(np.array(bounds, np.int32)), dw)
        assert np.array_equal(dw.float().cpu().numpy(), want if dtype is F32 else ref.bf16(want))


@pytest.mark.parametrize("M,N,variant", [(2048, 4096, "tile128x256"), (8000, 2000, "tile256x256")])
def test_rows_scales_whose_products_are_tiny_or_not_numbers(M, N, variant):
    """Scales by rows on both sides, whose products are subnormal in some blocks, huge, infinite or NaN in others: the large
    tiles, which let the matrix cores multiply them, give the bits of the kernel of few rows."""
    rng = np.random.default_rng(M)
    K, nb = 272, 3
    a, w = (dev(rng.integers(0, 0x7F, (n, K)).astype(np.uint8)) for n in (M, N))
    sa, sw = (dev((rng.random((n, nb)) * 2.0 ** rng.integers(-75, -60, (n, nb))).astype(np.float32)) for n in (M, N))
    sa[1::7] *= 2.0**125
    sw[::5] *= 2.0**125
    sa[3, 1], sa[9, 0], sw[4, 2], sw[6, 0] = float("nan"), float("inf"), float("nan"), 0.0
    y = torch.empty((M, N), device="cuda")
    mxmoe.fp8_block128_gemm(a, sa, w, sw, y)
    assert mxmoe.last_variant() == "b128:" + variant
    few = torch.empty((16, N), device="cuda")
    for m in (0, 16, M - 16):
        mxmoe.fp8_block128_gemm(a[m:m + 16], sa[m:m + 16], w, sw, few)
        assert torch.equal(few.nan_to_num(7.0), y[m:m + 16].nan_to_num(7.0)) and torch.equal(few.isnan(), y[m:m + 16].isnan())


@pytest.mark.parametrize("E,R,N,K,variant", [(16, 90, 60, 400, "rows16"), (16, 1000, 300, 656, "tile64x64"), (200, 900, 60, 144, "tile64x64"),
                                             (40, 70, 1100, 1040, "tile16x64"), (300, 600, 130, 272, "tile16x64"), (30, 60, 300, 144, "tile16x64"),
                                             (16, 1000, 1030, 272, "tile64x128"), (200, 1000, 300, 400, "tile64x128"),
                                             (16, 1600, 1500, 528, "tile128x256"), (1, 1300, 1500, 400, "tile64x128"),   # 21 x 12 workgroups
                                             (4, 6000, 1500, 400, "tile256x256"), (16, 20000, 300, 144, "tile256x256")])
def test_every_kernel_of_experts_in_order(E, R, N, K, variant):
    rng = np.random.default_rng(E + R + N)
    bounds = ragged(rng, E, R) if E > 1 else [0, R]
    a, a_sc = ref.whole_codes(rng, R, K), ref.short_scales(rng, R, blocks(K))
    w = ref.whole_codes(rng, E * N, K).reshape(E, N, K)
    w_sc = ref.short_scales(rng, E * blocks(N), blocks(K)).reshape(E, blocks(N), blocks(K))
    want = np.full((R, N), 7.0, np.float32)
    for e, (i, j) in enumerate(zip(bounds, bounds[1:])):
        if i < j:
            want[i:j] = ref.in_order(a[i:j], a_sc[i:j], w[e], w_sc[e], B)
    args = [dev(v) for v in (a, a_sc, w, w_sc)]
    assert np.array_equal(grouped(*args, bounds, F32).cpu().numpy(), want)
    assert mxmoe.last_variant() == "b128:" + variant
    assert np.array_equal(grouped(*args, bounds, BF16).float().cpu().numpy(), ref.bf16(want))


@pytest.mark.parametrize("E,rows,N,K,variant", [(8, 1500, 300, 270, "tile128x128"), (65, 6000, 300, 270, "tile256x256"),
                                                (20, 9000, 520, 513, "tile256x256")])
def test_every_kernel_of_weight_gradients_in_order(E, rows, N, K, variant):
    rng = np.random.default_rng(E + N)
    bounds = ragged(rng, E, rows)
    ld = mxmoe.fp8_quantize128_t_cols(rows, E)
    a, b = ref.whole_codes(rng, N, ld), ref.whole_codes(rng, K, ld)
    a_sc, b_sc = ref.short_scales(rng, N, ld // B), ref.short_scales(rng, K, ld // B)
    dw = torch.full((E, N, K), 7.0, device="cuda")
    mxmoe.fp8_block128_grouped_wgrad(*[dev(v) for v in (a, a_sc, b, b_sc)], dev(np.array(bounds, np.int32)), dw)
    assert mxmoe.last_variant() == "b128:" + variant
    at = 0
    for e, (i, j) in enumerate(zip(bounds, bounds[1:])):
        n = blocks(j - i)
        s, t = slice(at * B, (at + n) * B), slice(at, at + n)
        want = ref.in_order(a[:, s], a_sc[:, t], b[:, s], b_sc[:, t], 1) if n else np.zeros((N, K), np.float32)
        assert np.array_equal(dw[e].cpu().numpy(), want)
        at += n
