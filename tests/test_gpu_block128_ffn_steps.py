"""ExpertFFN128 is its steps, bit for bit, and each step is the 64-bit form of the one before."""
import numpy as np
import pytest
import torch

import block128_ref as ref
from block128_ref import BF16, F32, U8, B, blocks, dev, typed
from block_scaled_fp8xfp4_amd import mxmoe
from block_scaled_fp8xfp4_amd.layer import ExpertFFN128, Route, quantize128
from test_gpu_block128_layers import ffn_weights

pytestmark = pytest.mark.gpu


def host(t):
    return t.double().cpu().numpy()


def close(got, v, w):
    """The kept bf16 rows `got` against rows v times w^T: matrix cores cut 2^-10 of the sum of magnitudes at most, fp32 rounds
    once a block and scale, bf16 once.  Of their norm: the cut is 3.4e-5 (5e-5 with fp32's and the spread between rows); where it
    carries a value over a bf16 border the difference from the rounded exact one is a whole step, at most 2^-7 of the value, and
    half of one otherwise nothing.  A value is within 5e-5 of a border that lies 2^-8 apart or more with a probability of at
    most 2 * 5e-5 * 2^8 = 1 in 39, so the norm of the difference is at most 2^-7 / sqrt(39) = 1.25e-3 of the results'."""
    exact, most = v @ w.T, np.abs(v) @ np.abs(w).T
    cut = (2.0**-10 + (blocks(v.shape[1]) + 2) * 2.0**-23) * most
    assert (np.abs(got - exact) <= cut + 2.0**-8 * (np.abs(exact) + cut)).all()
    return np.square(got - ref.bf16(exact)).sum(), np.square(exact).sum()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,k,E,H,I,skip", [(1, 2, 8, 256, 128, False), (5, 3, 7, 272, 144, True), (40, 4, 16, 400, 208, True),
                                            (300, 2, 4, 512, 320, False)])
def test_expert_ffn_is_its_steps(T, k, E, H, I, skip, dtype):
    rng = np.random.default_rng(T)
    torch.manual_seed(T)
    (w13, s13), (w2, s2) = ffn_weights(rng, E, H, I)
    x, xv = typed(rng.standard_normal((T, H)), BF16)
    route = Route(T, E, k)
    route(torch.randn((T, E), device="cuda"), torch.rand(T, device="cuda") if skip else None, 0.3)
    R = T * k
    y = ExpertFFN128(*[dev(v) for v in (w13, s13, w2, s2)])(x, route, dtype=dtype)

    q, sc = quantize128(x)
    xs, xs_sc = torch.zeros((R, H), dtype=U8, device="cuda"), torch.ones((R, blocks(H)), device="cuda")
    mxmoe.moe_permute(q, route.slot_pos, xs, sc, xs_sc)
    gu = torch.zeros((R, 2 * I), dtype=BF16, device="cuda")
    mxmoe.fp8_block128_grouped_gemm(xs, xs_sc, dev(w13), dev(s13), route.offsets, gu)
    a, a_sc = torch.zeros((R, I), dtype=U8, device="cuda"), torch.ones((R, blocks(I)), device="cuda")
    mxmoe.fp8_swiglu_quantize128(gu, a, a_sc)
    o, y2 = torch.zeros((R, H), dtype=BF16, device="cuda"), torch.full((T, H), 7.0, dtype=dtype, device="cuda")
    mxmoe.fp8_block128_grouped_gemm(a, a_sc, dev(w2), dev(s2), route.offsets, o)
    mxmoe.moe_unpermute(o, route.w, route.slot_pos, y2)
    assert torch.equal(y, y2)

    want_q, want_sc = ref.cast(xv, 1, B)
    pos, off = route.slot_pos.cpu().numpy(), route.offsets.cpu().numpy()
    live, t = pos[pos >= 0], np.nonzero(pos >= 0)[0]
    assert np.array_equal(xs.cpu().numpy()[live], want_q[t]) and np.array_equal(xs_sc.cpu().numpy()[live], want_sc[t])
    guv, n = host(gu), off[E]
    act = (guv[:, :I] / (1 + np.exp(-guv[:, :I])) * guv[:, I:]).astype(np.float32).astype(np.float64)
    want_q, want_sc = ref.cast(act[:n], 1, B)
    assert np.array_equal(a.cpu().numpy()[:n], want_q) and np.array_equal(a_sc.cpu().numpy()[:n], want_sc)
    for got, v, w, w_sc in ((guv, ref.wide(xs.cpu().numpy(), xs_sc.cpu().numpy(), 1), w13, s13),
                            (host(o), ref.wide(a.cpu().numpy(), a_sc.cpu().numpy(), 1), w2, s2)):
        off2, norm2 = 0.0, 0.0
        for e in range(E):
            i, j = off[e], off[e + 1]
            if i < j:
                d = close(got[i:j], v[i:j], ref.wide(w[e], w_sc[e], B))
                off2, norm2 = off2 + d[0], norm2 + d[1]
        print(f"{np.sqrt(off2 / norm2):.2e} of the norm", flush=True)
        assert off2 <= 1.25e-3**2 * norm2
