"""Infinities and NaN in the casts with a scale for each block of 128: the block that holds one has the scale NaN, and every other
code and scale is as without it."""
import pytest
import torch

from block_scaled_fp8xfp4_amd import mxmoe

pytestmark = pytest.mark.gpu

BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
INF, NAN = float("inf"), float("nan")


def payload(low):
    """The fp32 NaN with these low bits and a quiet bit, and the one without (it looks like an infinity but for them)."""
    return [torch.tensor([bits | low], dtype=torch.int32).view(F32) for bits in (0x7FC00000, 0x7F800000)]


def only_that_block(q, sc, q0, sc0, row, block, cols):
    """sc is NaN at [row, block] alone; the other blocks' codes and scales are q0's and sc0's."""
    assert sc[row, block].isnan() and sc.isnan().sum() == 1
    same = ~sc.isnan()
    assert torch.equal(sc[same], sc0[same])
    keep = torch.ones_like(q, dtype=torch.bool)
    keep[row, cols] = False
    assert torch.equal(q[keep], q0[keep])


# (gate, up): what silu(gate) up is not finite for; None: as it is
PAIRS = [(INF, None), (None, INF), (None, -INF), (NAN, None), (None, NAN), (-INF, None), (INF, 0.0), (0.0, INF), (-200.0, INF),
         (1e30, 1e30), (-1e30, NAN), (80.0, -3.4e38)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,I", [(3, 144), (130, 1040)])
def test_swiglu(dtype, T, I):
    gu0 = (torch.randn((T, 2 * I), device="cuda") * 2).to(dtype)
    q0, sc0 = torch.zeros((T, I), dtype=U8, device="cuda"), torch.zeros((T, -(-I // 128)), device="cuda")
    mxmoe.fp8_swiglu_quantize128(gu0, q0, sc0)
    assert sc0.isfinite().all()
    for n, (g, u) in enumerate(PAIRS):
        for row, col in ((0, 0), (1, I - 1), (T - 1, n), (T // 2, 128 + n)):
            gu = gu0.clone()
            if g is not None:
                gu[row, col] = g
            if u is not None:
                gu[row, I + col] = u
            q, sc = torch.zeros_like(q0), torch.zeros_like(sc0)
            mxmoe.fp8_swiglu_quantize128(gu, q, sc)
            b = col // 128
            only_that_block(q, sc, q0, sc0, row, b, slice(b * 128, (b + 1) * 128))


@pytest.mark.parametrize("low", [1, 5, 7, 8])
def test_swiglu_of_nan_with_low_bits_alone(low):
    """The largest near values carry their places in three low bits: a NaN whose own bits are only there stays one."""
    T, I = 4, 272
    gu0 = torch.randn((T, 2 * I), device="cuda")
    q0, sc0 = torch.zeros((T, I), dtype=U8, device="cuda"), torch.zeros((T, 3), device="cuda")
    mxmoe.fp8_swiglu_quantize128(gu0, q0, sc0)
    for v in payload(low):
        for at, (row, col) in enumerate(((0, 0), (1, 7), (2, 271), (3, 200))):
            gu = gu0.clone()
            gu[row, col + (I if at % 2 else 0):][:1] = v.cuda()
            q, sc = torch.zeros_like(q0), torch.zeros_like(sc0)
            mxmoe.fp8_swiglu_quantize128(gu, q, sc)
            only_that_block(q, sc, q0, sc0, row, col // 128, slice(col // 128 * 128, col // 128 * 128 + 128))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bounds,cols", [([0, 300], 70), ([0, 0, 5, 5, 133, 400], 9), ([0, 200, 329], 130)])
def test_columns(dtype, bounds, cols):
    rows, E = bounds[-1], len(bounds) - 1
    src0 = torch.randn((rows, cols), device="cuda").to(dtype)
    off = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    ld = mxmoe.fp8_quantize128_t_cols(rows, E)

    def cast(src):
        q, sc = torch.zeros((cols, ld), dtype=U8, device="cuda"), torch.zeros((cols, ld // 128), device="cuda")
        mxmoe.fp8_quantize128_t(src, q, sc, off)
        return q, sc

    first, block_of = 0, {}
    for a, b in zip(bounds, bounds[1:]):
        for r in range(a, b):
            block_of[r] = first + (r - a) // 128
        first += -(-(b - a) // 128)
    q0, sc0 = cast(src0)
    bad = [torch.tensor([v]) for v in (INF, -INF, NAN)] + (payload(1) if dtype is F32 else [])
    for n, v in enumerate(bad):
        for row in (0, bounds[1] - 1 if bounds[1] else 4, rows - 1, rows // 2):      # and a group's last, partial block
            src, col = src0.clone(), (n * 31 + row) % cols
            src[row, col:col + 1] = v.to("cuda", dtype) if dtype is BF16 else v.cuda()
            q, sc = cast(src)
            b = block_of[row]
            only_that_block(q, sc, q0, sc0, col, b, slice(b * 128, (b + 1) * 128))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_rows_and_tiles(dtype, block_rows):
    rows, cols = 200, 304
    src0 = torch.randn((rows, cols), device="cuda").to(dtype)

    def cast(src):
        q, sc = torch.zeros((rows, cols), dtype=U8, device="cuda"), torch.zeros((-(-rows // block_rows), 3), device="cuda")
        mxmoe.fp8_quantize128(src, q, sc, block_rows)
        return q, sc

    q0, sc0 = cast(src0)
    bad = [torch.tensor([v]) for v in (INF, -INF, NAN)] + (payload(1) if dtype is F32 else [])
    for v in bad:
        for row, col in ((0, 0), (131, 130), (199, 303)):
            src = src0.clone()
            src[row, col:col + 1] = v.to("cuda", dtype) if dtype is BF16 else v.cuda()
            q, sc = cast(src)
            i, b = row // block_rows, col // 128
            assert sc[i, b].isnan() and sc.isnan().sum() == 1
            same = ~sc.isnan()
            keep = torch.ones_like(q, dtype=torch.bool)
            keep[i * block_rows:(i + 1) * block_rows, b * 128:(b + 1) * 128] = False
            assert torch.equal(sc[same], sc0[same]) and torch.equal(q[keep], q0[keep])
