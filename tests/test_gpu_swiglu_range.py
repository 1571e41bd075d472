"""The SwiGLU cast over the whole range of its finite inputs, in every kernel that makes it: mx_swiglu_quantize and the
gate/up products of fp4_dense_ffn.

Codes and scales are those of silu(gate) * up in 64 bits rounded once to fp32, bit for bit: no tolerance.  The kernels
take them from a short fp32 evaluation where that decides them, so these inputs sit where fp32 leaves its range inside the
evaluation: gates near the type's largest value (gate * log2 e overflows from 2.36e38 on) and under its smallest normal value
(half of them loses bits), with ups that bring the product back to the size of ordinary neighbours."""
import numpy as np
import pytest
import torch

import dense_block_ref as ref
from block_scaled_fp8xfp4_amd import mxmoe
from dense_block_ref import E2M1, E4M3, codes_like, to_dev
from gpu_common import host, say
from test_gpu_dense_block import same_bits, typed

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HUGE = [2.3e38, 2.35e38, 2.37e38, 2.4e38, 3e38, 3.3e38, 3.38e38]


def cast(gu, fmt):
    q, sc = codes_like(gu.shape[0], gu.shape[1] // 2, fmt)
    mxmoe.mx_swiglu_quantize(gu, q, sc, fmt)
    return q, sc


def one_gate_per_block(gates, ups, blocks):
    """Rows [1, 2 * 32 * blocks]: ordinary values, and one of the (gate, up) pairs in a place of its own in each block."""
    rng = np.random.default_rng(blocks)
    g = rng.standard_normal((1, 32 * blocks)).astype(np.float32)
    u = rng.standard_normal((1, 32 * blocks)).astype(np.float32)
    for b in range(blocks):
        g[0, 32 * b + (7 * b) % 32] = gates[b % len(gates)]
        u[0, 32 * b + (7 * b) % 32] = ups[b % len(ups)]
    return np.concatenate([g, u], -1)


@pytest.mark.parametrize("fmt", [E4M3, E2M1])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gates_near_the_largest_value(dtype, fmt):
    """Huge gates among ordinary ones: the products from far below to far above their neighbours."""
    ups = [1e-30, -1e-38, 4e-39, -1e-45, 0.0, 1e-33, -1.0, 1e-40, 3e-37]        # 7 gates by 9 ups: every pair in 63 blocks
    with np.errstate(over="ignore"):
        t, v = typed(one_gate_per_block(HUGE, ups, 63), dtype)
        q, sc = cast(t, fmt)
        rq, rs = ref.quantize(ref.swiglu(v), fmt)
    same_bits(sc, rs, "scales")
    same_bits(q, rq, "codes")


@pytest.mark.parametrize("fmt", [E4M3, E2M1])
def test_gates_under_the_smallest_normal_value(fmt):
    """Blocks of gates of a few units of 2^-149, and up to 2^-120, that large ups bring back."""
    rng = np.random.default_rng(4)
    g = (rng.integers(1, 16, (40, 32)) * 2.0 ** -149).astype(np.float32)
    g[20:] = (rng.standard_normal((20, 32)) * 2.0 ** rng.integers(-140, -119, (20, 1))).astype(np.float32)
    u = (rng.choice([-1.0, 1.0], (40, 32)) * rng.uniform(1, 2, (40, 32)) * 2.0 ** rng.integers(118, 124, (40, 32))).astype(np.float32)
    gu = np.concatenate([g, u], -1)
    q, sc = cast(to_dev(gu), fmt)
    rq, rs = ref.quantize(ref.swiglu(gu), fmt)
    same_bits(sc, rs, "scales")
    same_bits(q, rq, "codes")


@pytest.mark.parametrize("fmt", [E4M3, E2M1])
def test_a_row_alone_and_beside_one_that_needs_double(fmt):
    """A row with huge gates has the same codes alone and beside a row of gates far below zero, which sends the
    wavefront that both share to the evaluation in double."""
    I = 64                                                             # eight rows to a wavefront
    gu = one_gate_per_block([3e38, 2.4e38], [1e-30, -1e-30], 2)
    alone = cast(to_dev(gu), fmt)
    both = np.concatenate([gu, np.full_like(gu, -80.0), gu], 0)
    q, sc = cast(to_dev(both), fmt)
    for r in (0, 2):
        assert torch.equal(q[r], alone[0][0]) and torch.equal(sc[r], alone[1][0]), r
    same_bits(q[0], ref.quantize(ref.swiglu(gu), fmt)[0][0], "codes")


# The kernels of the gate/up product: the (T, H, I) of test_fp4_dense_ffn_blocks_that_need_double, and one row.
FFN_SIZES = [(1, 256, 64), (5, 256, 96), (40, 256, 96), (40, 128, 4128), (600, 128, 1056), (1100, 160, 2080),
             (1500, 128, 2080), (2040, 544, 4064), (2100, 256, 4128), (8, 2048, 256)]


def check_ffn(T, H, I, fmt, scales, last_scale, alone=False):
    """The FFN of rows with far columns (two or three in each block of the intermediate) among ordinary ones against the
    64-bit cast of its gate/up values and the product of that.  The far columns read one element of a row each: the first
    of its first block for the gate, of its second for the up; the ordinary columns read the row's other blocks.
    scales: exponents of the first block of the rows, and of the far gates (even, odd) and ups; last_scale: of the first
    block of the last row, whose ordinary columns are zeros with alone.  Returns the gate/up values."""
    rng = np.random.default_rng(T + I)
    half, one = (32, 0x38) if fmt == E4M3 else (16, 2)                 # bytes of a block, the code of 1.0
    x, x_sc = ref.quantize(ref.activations(rng, T, H), fmt)
    w13, w13_sc = ref.weights(rng, 2 * I, H)
    row, even, odd, up = scales
    x[:, :2 * half] = 0
    x[:, 0] = x[:, half] = one
    if alone:
        x[T - 1, 2 * half:] = 0
    x_sc[:, 0], x_sc[:, 1], x_sc[T - 1, 0] = 127 + row, 127, 127 + last_scale
    w13[:, :32] = 0
    far = np.arange(0, I, 11)
    w13[far], w13[I + far] = 0, 0
    w13[far, 0], w13[I + far, 16] = 3, 3                               # 1.5
    w13_sc[far, 0] = 127 + np.where(far % 2 == 0, even, odd)
    w13_sc[I + far, 1] = 127 + up
    w2, w2_sc = ref.weights(rng, H, I)
    x, x_sc, w13, w13_sc, w2, w2_sc = (to_dev(t) for t in (x, x_sc, w13, w13_sc, w2, w2_sc))
    gu = torch.empty((T, 2 * I), dtype=F32, device="cuda")
    mxmoe.fp4_block_gemm(x, x_sc, fmt, w13, w13_sc, gu)
    v = host(gu)
    rq, rs = ref.quantize(ref.swiglu(v), fmt)
    want = torch.empty((T, H), dtype=F32, device="cuda")
    mxmoe.fp4_block_gemm(to_dev(rq), to_dev(rs), fmt, w2, w2_sc, want)
    ws = torch.empty(mxmoe.fp4_dense_ffn_workspace_bytes(T, H, I, fmt), dtype=torch.uint8, device="cuda")
    y = torch.empty((T, H), dtype=F32, device="cuda")
    mxmoe.fp4_dense_ffn(x, x_sc, fmt, w13, w13_sc, w2, w2_sc, fmt, y, ws)
    assert torch.equal(y.view(torch.int32), want.view(torch.int32)), mxmoe.last_variant()
    say(f"{mxmoe.last_variant()}: T {T} H {H} I {I}")
    return v


@pytest.mark.parametrize("fmt", [E4M3, E2M1])
@pytest.mark.parametrize("T,H,I", FFN_SIZES)
def test_ffn_gates_near_the_largest_value(T, H, I, fmt):
    """Gates of 1.5 * 2^127 (2.55e38) and 1.5 * 2^126 that ups of 1.5 * 2^-107 bring back, in every kernel of the gate/up
    product; the last row's are 2^-8 of that."""
    v = check_ffn(T, H, I, fmt, (63, 64, 63, -107), 63 if T == 1 else 55)
    assert v[:, :I].max() == np.float32(1.5 * 2.0 ** 127)


def every_gate(fmt, sign, lo, hi):
    """Every fp32 gate with magnitude bits in [lo, hi), each with an up that brings the product to between 2^-9 and 2^6
    where one exists, against the 64-bit form on the GPU and mx_quantize."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(fmt)
    n, cols = 1 << 25, 2048
    for first in range(lo, hi, n):
        b = torch.arange(first, min(first + n, hi), dtype=torch.int32, device="cuda")
        g = (b | -2 ** 31 if sign else b).view(F32).view(cols, -1).t().contiguous()   # a block's gates lie far apart
        s = g.double()
        s = s / (1 + torch.exp(-s))
        r = torch.exp2(torch.rand(g.shape, generator=gen, device="cuda") * 15 - 9)
        r = torch.where(torch.rand(g.shape, generator=gen, device="cuda") < 0.5, r, -r)
        u = (r.double() / s).nan_to_num(0.0).clamp(-3.4e38, 3.4e38).float()
        a = (s * u.double()).float()
        want_q, want_s = codes_like(*g.shape, fmt)
        mxmoe.mx_quantize(a, want_q, want_s, fmt)
        q, sc = cast(torch.cat([g, u], -1), fmt)
        wrong = int((q != want_q).sum()) + int((sc != want_s).sum())
        assert wrong == 0, f"{wrong} bytes differ, gates from {hex(first)} on"


@pytest.mark.parametrize("fmt", [E4M3, E2M1])
def test_every_normal_gate(fmt):
    """From 2^-120 to the largest float, and to -60 (below, the kernels use the double form)."""
    every_gate(fmt, 0, 0x03800000, 0x7F800000)
    every_gate(fmt, 1, 0x03800000, 0x42700000)


@pytest.mark.parametrize("fmt", [E4M3, E2M1])
@pytest.mark.parametrize("T,H,I", FFN_SIZES)
def test_ffn_gates_under_the_smallest_normal_value(T, H, I, fmt):
    """A last row of gates of 3 and 6 units of 2^-149 alone, with ups of 1.5 * 2^120, in every kernel of the gate/up product:
    half of 3 units is no float."""
    v = check_ffn(T, H, I, fmt, (63, -76, -75, 120), -72, alone=True)
    assert v[T - 1, 0] == np.float32(3 * 2.0 ** -149) and v[T - 1, I] == np.float32(1.5 * 2.0 ** 120)


@pytest.mark.parametrize("fmt", [E4M3, E2M1])
def test_every_subnormal_gate(fmt):
    """To 2^-120, both signs."""
    every_gate(fmt, 0, 0, 0x03800000)
    every_gate(fmt, 1, 0, 0x03800000)
