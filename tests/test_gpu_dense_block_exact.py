"""The dense block's products and casts held to what their arithmetic allows, where a wrong or missing element would show.

E4M3 x E2M1 on the matrix cores (measured on MI355X).  Of every eight consecutive K, with E the largest sum of the two
operands' exponents among their products that are not zero (a subnormal counts as the format's smallest exponent), each
product is cut toward zero to a multiple of 2^(E - 13) under the block's scales.  Then a step of 64 joins the eight sums
and the accumulator, each cut below 2^-24 of the largest, and rounds once.  So with `lost` the parts that are cut, summed
over a row's products, and A = sum |a w|, a result of S = ceil(K / 64) steps is off by at most
    lost + S (9 + 1) 2^-24 A = lost + 5 S 2^-23 A.
Products of small whole numbers under few scales lose nothing and their sums fit 24 bits: those results are exact.  A bf16
result is the fp32 one rounded, at most 2^-8 of it more."""
import numpy as np
import pytest
import torch

import dense_block_ref as ref
from block_scaled_fp8xfp4_amd import mxmoe
from dense_block_ref import E2M1, E4M3, codes_like, to_dev
from gpu_common import host, say
from test_gpu_dense_block import random_codes, same_bits

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
ONE = 127


def pack(values, fmt):
    """Numbers that the format has -> code bytes."""
    t = torch.from_numpy(values)
    if fmt == E4M3:
        return t.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    c = torch.bucketize(t.abs(), mids).to(torch.uint8) | (torch.signbit(t).to(torch.uint8) << 3)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).numpy()


def whole_numbers(rng, rows, K, fmt, scales):
    """Elements of +-{0, 1, 2, 3, 4, 6} (and 5, 7, 8 in E4M3) under scales drawn per block: (codes, scales, values)."""
    most = [0, 1, 2, 3, 4, 6] + ([5, 7, 8] if fmt == E4M3 else [])
    v = (rng.choice(most, (rows, K)) * rng.choice([-1.0, 1.0], (rows, K))).astype(np.float32)
    sc = rng.choice(scales, (rows, K // 32)).astype(np.uint8)
    q = pack(v, fmt)
    return q, sc, ref.values(q, sc, fmt)


# few rows alone, through LDS, and by sixteens; tiles of 32 x 64, 64 x 64, 128 x 128, 128 x 256, 256 x 256; K to every end
EXACT_SIZES = [(1, 16, 32), (1, 4096, 4096), (3, 40, 544), (16, 72, 1056), (16, 16400, 512), (2, 40, 16384), (33, 1152, 256),
               (40, 2801, 640), (64, 130, 2080), (129, 40, 16384), (300, 520, 992), (1040, 523, 1056), (1500, 1502, 4096),
               (2100, 2835, 1184), (2830, 2835, 512)]


@pytest.mark.parametrize("fmt", [E4M3, E2M1])
@pytest.mark.parametrize("M,N,K", EXACT_SIZES)
def test_products_of_whole_numbers_are_exact(M, N, K, fmt):
    """Products are multiples of the smallest scales' product and at most 48 of it (times 16 where scales differ: K of 4096
    at most), their sums under 2^24 of it: equal to the 64-bit product."""
    rng = np.random.default_rng(M + N + K)
    scales = (ONE, ONE + 1, ONE + 2) if K <= 4096 else (ONE,)
    a, a_sc, av = whole_numbers(rng, M, K, fmt, scales)
    w, w_sc, wv = whole_numbers(rng, N, K, E2M1, scales)
    assert K * 48 * (16 if len(scales) > 1 else 1) < 2 ** 24
    want = to_dev(av) @ to_dev(wv).t().contiguous()                    # whole numbers in 64 bits: exact
    d = [to_dev(t) for t in (a, a_sc, w, w_sc)]
    y32, y16 = (torch.empty((M, N), dtype=t, device="cuda") for t in (F32, BF16))
    mxmoe.fp4_block_gemm(d[0], d[1], fmt, d[2], d[3], y32)
    v = mxmoe.last_variant()
    mxmoe.fp4_block_gemm(d[0], d[1], fmt, d[2], d[3], y16)
    assert torch.equal(y32.double(), want), v
    assert torch.equal(y16, y32.to(BF16)), v
    say(f"{v}: {M} x {N} x {K}")


def exponents(v, least):
    """The exponent of each value, at least the format's smallest; very small for zeros."""
    e = np.frexp(np.abs(v))[1] - 1
    return np.where(v == 0, -1000, np.maximum(e, least))


def product_and_room(a, a_sc, w, w_sc):
    """(the 64-bit product, how far the matrix cores' may be from it) of E4M3 rows a and E2M1 rows w."""
    M, N, K = a.shape[0], w.shape[0], a.shape[1]
    plain = np.full_like(a_sc, ONE), np.full_like(w_sc, ONE)
    ae, we = ref.values(a, plain[0], E4M3), ref.values(w, plain[1], E2M1)
    ax, wx = exponents(ae, -6), exponents(we, 0)
    y, room = np.empty((M, N)), np.empty((M, N))
    S = -(-K // 64)
    for m in range(M):
        p = ae[m] * we                                                 # [N, K]: the elements' products
        E = (ax[m] + wx).reshape(N, K // 8, 8).max(-1).repeat(8, -1)
        q = np.ldexp(1.0, np.maximum(E, -200) - 13)
        lost = np.abs(p) - np.floor(np.abs(p) / q) * q
        x = np.ldexp(1.0, a_sc[m].astype(int) + w_sc.astype(int) - 2 * ONE).repeat(32, -1)
        y[m] = (p * x).sum(-1)
        room[m] = (lost * x).sum(-1) + 5 * S * 2.0 ** -23 * (np.abs(p) * x).sum(-1)
    return y, room


@pytest.mark.parametrize("kind", ["normal", "any codes", "wide scales"])
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (1, 96, 576), (7, 40, 544), (16, 72, 1056), (48, 2049, 4096), (64, 130, 2080),
                                   (300, 520, 992), (1040, 523, 1056), (1500, 1502, 4096), (2830, 2835, 576)])
def test_e4m3_products_lose_no_more_than_the_instruction_cuts(M, N, K, kind):
    rng = np.random.default_rng(M + N + K)
    if kind == "normal":
        a, a_sc = ref.quantize(ref.activations(rng, M, K), E4M3)
        w, w_sc = ref.weights(rng, N, K)
    else:
        a, a_sc = random_codes(rng, M, K, E4M3)
        w, w_sc = random_codes(rng, N, K, E2M1)
        if kind == "wide scales":
            a_sc, w_sc = (rng.integers(100, 155, s.shape).astype(np.uint8) for s in (a_sc, w_sc))
    d = [to_dev(t) for t in (a, a_sc, w, w_sc)]
    y32 = torch.empty((M, N), dtype=F32, device="cuda")
    mxmoe.fp4_block_gemm(d[0], d[1], E4M3, d[2], d[3], y32)
    rows = np.unique(np.concatenate([[0, M - 1], rng.integers(0, M, 10)]))      # some rows and columns of them
    cols = np.unique(np.concatenate([[0, N - 1], rng.integers(0, N, 60)]))
    want, room = product_and_room(a[rows], a_sc[rows], w[cols], w_sc[cols])
    over = np.abs(host(y32).astype(np.float64)[np.ix_(rows, cols)] - want) - room
    assert over.max() <= 0, f"{mxmoe.last_variant()}: {over.max():.3e} more than the bound"
    say(f"{mxmoe.last_variant()}: off by at most {(over + room).max() / np.abs(want).max():.1e} of the largest")


@pytest.mark.parametrize("T,H,I", [(1, 4096, 576), (2, 512, 2048), (5, 256, 96), (16, 4096, 2048), (48, 4096, 576), (40, 128, 4128),
                                   (600, 128, 1056), (1100, 160, 2080), (1500, 128, 2080), (2100, 256, 4128)])
def test_e4m3_ffn_against_its_64_bit_form(T, H, I):
    """Rows and gate/up weights of whole numbers, whose products are exact, so the intermediate's codes are those of the
    64-bit form; then the second product within what the instruction cuts.  In every kernel of the gate/up product."""
    rng = np.random.default_rng(T + H + I)
    x, _, xv = whole_numbers(rng, T, H, E4M3, (ONE,))
    w13, _, wv = whole_numbers(rng, 2 * I, H, E2M1, (ONE,))
    down = int(np.ceil(np.log2(np.sqrt(H) * 13 / 2)))                  # gates and ups of about 2
    x_sc = np.full((T, H // 32), ONE - down, np.uint8)
    w13_sc = np.full((2 * I, H // 32), ONE, np.uint8)
    w2, w2_sc = ref.weights(rng, H, I)
    gu = host((to_dev(xv) @ to_dev(wv).t().contiguous()) * 2.0 ** -down).astype(np.float32)
    q, sc = ref.quantize(ref.swiglu(gu), E4M3)
    ws = torch.empty(mxmoe.fp4_dense_ffn_workspace_bytes(T, H, I, E4M3), dtype=torch.uint8, device="cuda")
    y32, y16 = (torch.empty((T, H), dtype=t, device="cuda") for t in (F32, BF16))
    d = [to_dev(t) for t in (x, x_sc, w13, w13_sc, w2, w2_sc)]
    for y in (y32, y16):
        mxmoe.fp4_dense_ffn(d[0], d[1], E4M3, *d[2:], E4M3, y, ws)
    rows = np.unique(np.concatenate([[0, T - 1], rng.integers(0, T, 10)]))
    cols = np.unique(np.concatenate([[0, H - 1], rng.integers(0, H, 60)]))
    want, room = product_and_room(q[rows], sc[rows], w2[cols], w2_sc[cols])
    over = np.abs(host(y32).astype(np.float64)[np.ix_(rows, cols)] - want) - room
    assert over.max() <= 0, f"{mxmoe.last_variant()}: {over.max():.3e} more than the bound"
    assert torch.equal(y16, y32.to(BF16))
    say(f"{mxmoe.last_variant()}: T {T} H {H} I {I}")


@pytest.mark.parametrize("fmt", [E4M3, E2M1])
@pytest.mark.parametrize("N,K", [(4096, 4096), (520, 992)])
def test_rows_past_the_largest_float_do_not_depend_on_M(N, K, fmt):
    """Finite operands whose sums pass fp32's largest value: infinities and NaN, the same bits alone and in every batch."""
    rng = np.random.default_rng(N)
    M = 600
    a, a_sc = random_codes(rng, M, K, fmt)
    w, w_sc = random_codes(rng, N, K, E2M1)
    a_sc[::2] = rng.integers(245, 255, a_sc[::2].shape)
    a, a_sc, w, w_sc = (to_dev(t) for t in (a, a_sc, w, w_sc))
    for dtype, bits in ((F32, torch.int32), (BF16, torch.int16)):
        whole = torch.empty((M, N), dtype=dtype, device="cuda")
        mxmoe.fp4_block_gemm(a, a_sc, fmt, w, w_sc, whole)
        assert torch.isinf(whole).any()
        for m in (1, 3, 16, 33, 64, 129, 320):
            y = torch.empty((m, N), dtype=dtype, device="cuda")
            mxmoe.fp4_block_gemm(a[:m], a_sc[:m], fmt, w, w_sc, y)
            assert torch.equal(y.view(bits), whole[:m].view(bits)), (m, dtype, mxmoe.last_variant())


# ----------------------------------------------------------- every float
def test_bf16_rounding_of_every_float():
    """The residual stream's rounding to bf16, of every fp32 value but NaN (through the addition alone)."""
    n, H = 1 << 26, 16384
    for first in range(-2 ** 31, 2 ** 31, n):
        x = torch.arange(first, first + n, dtype=torch.int64, device="cuda").to(torch.int32).view(F32)
        x = torch.where(torch.isnan(x), 0.0, x).view(-1, H)
        h = torch.empty_like(x, dtype=BF16)
        mxmoe.mx_add_rmsnorm(x, None, 1e-6, h=h)
        assert torch.equal(h.view(torch.int16), x.to(BF16).view(torch.int16)), hex(first & 0xFFFFFFFF)


@pytest.mark.parametrize("double", [False, True])
@pytest.mark.parametrize("fmt", [E4M3, E2M1])
def test_codes_of_every_float(fmt, double):
    """The SwiGLU cast's codes of every value from 2^-120 of a block's largest up against mx_quantize's: from the short form
    where that decides them, or from the double one (a block of gates under -60 in every wavefront, which holds 512
    columns).  silu(64) is 64, so an up of v gives 64 v, exactly; a block's first element is the format's largest value."""
    top, binade, scale = (448.0, 512.0, 2.0 ** 20) if fmt == E4M3 else (6.0, 8.0, 2.0 ** 20)
    rows, per_row = 1 << 16, 15 * 31
    end = int(np.float32(binade * scale / 64).view(np.int32))
    g = torch.full((rows, 16, 32), 64.0, device="cuda")
    if double:
        g[:, 0] = -61.0
    u = torch.ones((rows, 16, 32), device="cuda")
    u[:, 1:, 0] = top * scale / 64
    for sign in (1.0, -1.0):
        for first in range(0, end, rows * per_row):
            v = torch.arange(first, first + rows * per_row, dtype=torch.int32, device="cuda").clamp_(max=end - 1)
            u[:, 1:, 1:] = v.view(F32).view(rows, 15, 31) * sign
            q, sc = codes_like(rows, 512, fmt)
            want_q, want_s = codes_like(rows, 512, fmt)
            mxmoe.mx_swiglu_quantize(torch.cat([g.view(rows, 512), u.view(rows, 512)], -1), q, sc, fmt)
            mxmoe.mx_quantize((64.0 * u).view(rows, 512), want_q, want_s, fmt)
            wide = 32 if fmt == E4M3 else 16
            assert torch.equal(sc[:, 1:], want_s[:, 1:]), (sign, hex(first))
            assert torch.equal(q[:, wide:], want_q[:, wide:]), (sign, hex(first))
