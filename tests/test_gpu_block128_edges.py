"""Calls at the ends of what the experts' tokens and block-128 operators take: rows of few bytes, matrices whose rows lie apart,
room behind the results, all rows with one expert, the longest sums, as many threads as a call may have."""
import numpy as np
import pytest
import torch

import block128_ref as ref
from block128_ref import BF16, F32, U8, B, blocks, dev, plan, typed
from block_scaled_fp8xfp4_amd import mxmoe
from test_gpu_block128 import gemm, grouped, loud
from test_gpu_block128_far import codes, scales

pytestmark = pytest.mark.gpu


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("dtype,n", [(F32, 1), (F32, 3), (F32, 4), (U8, 1), (U8, 7), (U8, 15), (U8, 16), (U8, 33), (BF16, 9)])
def test_permute_with_few_scales(dtype, n):
    T, k, E, H = 37, 3, 9, 48
    slot_pos, _ = plan(np.random.default_rng(n), T, k, E, 0.8)
    x, sc = torch.randint(0, 255, (T, H), dtype=U8, device="cuda"), torch.randint(-90, 90, (T, n), device="cuda").to(dtype)
    out, out_sc = torch.full((T * k, H), 7, dtype=U8, device="cuda"), torch.full((T * k, n), 7, dtype=dtype, device="cuda")
    mxmoe.moe_permute(x, dev(slot_pos), out, sc, out_sc)
    want, want_sc = torch.full_like(out, 7), torch.full_like(out_sc, 7)
    for t, j in zip(*np.nonzero(slot_pos >= 0)):
        want[slot_pos[t, j]], want_sc[slot_pos[t, j]] = x[t], sc[t]
    assert torch.equal(out, want) and torch.equal(out_sc, want_sc)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_matrices_whose_rows_lie_apart(dtype, block_rows):
    """The C-ABI's row stride with several matrices: they follow one another at that stride."""
    n, rows, cols, ld = 3, 150, 208, 232
    src, v = typed(loud(np.random.default_rng(3), n * rows, ld), dtype)
    q = torch.full((n, rows, cols), 0xA5, dtype=U8, device="cuda")
    sc = torch.full((n, rows if block_rows == 1 else blocks(rows), blocks(cols)), -1.0, device="cuda")
    assert mxmoe.load().fp8_quantize128(src.data_ptr(), mxmoe.MX_IN_F32 if dtype is F32 else mxmoe.MX_IN_BF16, ld, n, rows, cols,
                                        block_rows, q.data_ptr(), sc.data_ptr(), stream()) == mxmoe.MX_OK
    for e in range(n):
        want_q, want_sc = ref.cast(v[e * rows:(e + 1) * rows, :cols], block_rows, B)
        assert np.array_equal(q[e].cpu().numpy(), want_q) and np.array_equal(sc[e].cpu().numpy(), want_sc)


@pytest.mark.parametrize("offsets", [False, True])
def test_columns_with_room_behind_them(offsets):
    """q wider than it has to be: what lies behind the last group is left as it was."""
    rows, cols, ld = 300, 70, 1024
    src, v = typed(loud(np.random.default_rng(4), rows, cols), BF16)
    q, sc = torch.full((cols, ld), 0xA5, dtype=U8, device="cuda"), torch.full((cols, ld // B), -1.0, device="cuda")
    mxmoe.fp8_quantize128_t(src, q, sc, torch.tensor([0, rows], dtype=torch.int32, device="cuda") if offsets else None)
    want_q, want_sc, _ = ref.columns(v, [0, rows], 384)
    assert np.array_equal(q[:, :384].cpu().numpy(), want_q) and np.array_equal(sc[:, :3].cpu().numpy(), want_sc)
    assert (q[:, 384:] == 0xA5).all() and (sc[:, 3:] == -1).all()


@pytest.mark.parametrize("E", [7, 256, 1024])
@pytest.mark.parametrize("R,N,K", [(3, 130, 144), (600, 130, 272), (5000, 520, 400)])
def test_all_rows_with_one_expert(E, R, N, K):
    rng = np.random.default_rng(E + R)
    a, a_sc = [dev(t) for t in ref.cast(loud(rng, R, K), 1, B)]
    w, w_sc = codes(E, N, K), scales(E, blocks(N), blocks(K))
    for e in (0, E // 2, E - 1):
        bounds = [0] * (e + 1) + [R] * (E - e)
        assert torch.equal(grouped(a, a_sc, w, w_sc, bounds, F32), gemm(a, a_sc, w[e], w_sc[e], F32)), e


@pytest.mark.parametrize("E,N,K", [(3, 100, 130), (300, 60, 70)])
def test_all_tokens_with_one_expert(E, N, K):
    rows = 700
    ld = mxmoe.fp8_quantize128_t_cols(rows, E)
    a, a_sc, b, b_sc = codes(N, ld), scales(N, ld // B), codes(K, ld), scales(K, ld // B)
    for e in (0, E // 2, E - 1):
        off = torch.tensor([0] * (e + 1) + [rows] * (E - e), dtype=torch.int32, device="cuda")
        dw = torch.full((E, N, K), 7.0, device="cuda")
        mxmoe.fp8_block128_grouped_wgrad(a, a_sc, b, b_sc, off, dw)
        n = blocks(rows)
        want = gemm(a[:, :n * B].contiguous(), a_sc[:, :n].contiguous(), b[:, :n * B].contiguous(), b_sc[:, :n].contiguous(), F32)
        assert torch.equal(dw[e], want) and dw.count_nonzero() == want.count_nonzero(), e


@pytest.mark.parametrize("M,N,w_rows", [(1, 16, 128), (20, 40, 1), (300, 300, 128)])
def test_longest_sums(M, N, w_rows):
    """K = 2^23, the most: a row's end against a sum of its last blocks alone, since the first ones are zeros."""
    K, tail = 1 << 23, 1 << 12
    a, w = torch.zeros((M, K), dtype=U8, device="cuda"), torch.zeros((N, K), dtype=U8, device="cuda")
    a[:, -tail:], w[:, -tail:] = codes(M, tail), codes(N, tail)
    a[:, :128], w[:, :128] = codes(M, 128), codes(N, 128)
    a_sc, w_sc = scales(M, K // B), scales(-(-N // w_rows), K // B)
    y = gemm(a, a_sc, w, w_sc, F32)

    def ends(t):
        return torch.cat([t[:, :128], t[:, -tail:]], 1)

    def ends_sc(t):
        return torch.cat([t[:, :1], t[:, -tail // B:]], 1)
    assert torch.equal(y, gemm(ends(a), ends_sc(a_sc), ends(w), ends_sc(w_sc), F32))       # zeros add nothing: acc = fma(0, s, acc)


def test_weight_gradients_of_the_most_tokens():
    """ld = 2^23 and tiles of 256 rows: the farthest byte of a tile lies 255 * 2^23 from its first."""
    E, N, ld = 100, 256, 1 << 23
    per = ld // E // B * B - 5
    a, a_sc, b, b_sc = codes(N, ld), scales(N, ld // B), codes(N, ld), scales(N, ld // B)
    off = (torch.arange(E + 1, device="cuda") * per).int()
    dw = torch.empty((E, N, N), device="cuda")
    mxmoe.fp8_block128_grouped_wgrad(a, a_sc, b, b_sc, off, dw)
    assert mxmoe.last_variant() == "b128:tile256x256"
    n = blocks(per)
    for e in (0, E // 2, E - 1):
        s, t = slice(e * n * B, (e + 1) * n * B), slice(e * n, (e + 1) * n)
        assert torch.equal(dw[e], gemm(a[:, s].contiguous(), a_sc[:, t].contiguous(), b[:, s].contiguous(), b_sc[:, t].contiguous(), F32))


def test_as_many_threads_as_a_call_may_have():
    """2^31 pieces of 16 bytes, 2^31 / 16 blocks, 2^31 columns of tokens, 2^24 slots."""
    T, row = 1 << 21, 1 << 14
    x = torch.empty((T, row), dtype=U8, device="cuda")               # 34 GB
    at = torch.tensor([0, 1, T // 2, T - 1], device="cuda")
    x[at] = torch.randint(0, 255, (4, row), dtype=U8, device="cuda")
    pos = torch.full((T, 1), -1, dtype=torch.int32, device="cuda")
    pos[at, 0] = torch.tensor([2, 0, 3, 1], dtype=torch.int32, device="cuda")
    out = torch.zeros((4, row), dtype=U8, device="cuda")
    mxmoe.moe_permute(x, pos, out)
    assert torch.equal(out[[2, 0, 3, 1]], x[at])
    del x, pos
    o, H = torch.randn((5, 1024), device="cuda").to(BF16), 1024
    pos = (torch.arange(T, device="cuda") % 6 - 1).int().view(T, 1)
    y = torch.empty((T, H), dtype=BF16, device="cuda")
    mxmoe.moe_unpermute(o, None, pos, y)
    want = torch.cat([torch.zeros_like(o[:1]), o])
    for r in (0, T // 2, T - 6):
        assert torch.equal(y[r:r + 6], want[(torch.arange(r, r + 6, device="cuda") % 6)])
    del y
    T, k, H = 1 << 20, 16, 9
    o, dy, w = torch.randn((T * k, H), device="cuda"), torch.randn((T, H), device="cuda"), torch.rand((T, k), device="cuda")
    pos = torch.arange(T * k, dtype=torch.int32, device="cuda").flip(0).view(T, k)
    d_o, dw = torch.empty_like(o), torch.empty_like(w)
    mxmoe.moe_unpermute_grad(dy, o, w, pos, d_o, dw)
    assert torch.equal(d_o.flip(0).view(T, k, H), dy[:, None] * w[:, :, None])
    far = torch.cat([torch.arange(50), torch.arange(T - 50, T)]).cuda()
    mine = o[pos[far].long()].double()
    assert ((dw[far].double() - (mine * dy[far, None].double()).sum(-1)).abs() <=
            15 * 2.0**-24 * (mine.abs() * dy[far, None].double().abs()).sum(-1)).all()
    del o, dy, w, pos, d_o, dw
    rows = 1 << 27
    src = torch.randn((rows, 16), device="cuda", dtype=BF16)
    q, sc = torch.empty((rows, 16), dtype=U8, device="cuda"), torch.empty((rows, 1), device="cuda")
    mxmoe.fp8_quantize128(src, q, sc)
    for r in (0, rows // 2, rows - 100):
        q1, sc1 = torch.empty((100, 16), dtype=U8, device="cuda"), torch.empty((100, 1), device="cuda")
        mxmoe.fp8_quantize128(src[r:r + 100], q1, sc1)
        assert torch.equal(q[r:r + 100], q1) and torch.equal(sc[r:r + 100], sc1)
