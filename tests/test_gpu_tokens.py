"""moe_permute, moe_unpermute and its gradient against 64-bit forms."""
import numpy as np
import pytest
import torch

import block128_ref as ref
from block128_ref import BF16, F32, U8, dev, plan, typed
from block_scaled_fp8xfp4_amd import mxmoe

pytestmark = pytest.mark.gpu

CASES = [(1, 1, 1, 1.0), (1, 8, 8, 1.0), (5, 3, 7, 0.6), (48, 8, 256, 0.8), (257, 2, 16, 1.0), (33, 16, 40, 0.5), (7, 4, 1024, 0.0)]


@pytest.mark.parametrize("T,k,E,live", CASES)
@pytest.mark.parametrize("dtype,H", [(U8, 1), (U8, 15), (U8, 16), (U8, 17), (U8, 4096), (BF16, 1), (BF16, 7), (BF16, 33),
                                     (BF16, 2050), (F32, 3), (F32, 5), (F32, 576), (torch.int64, 9)])
def test_permute(T, k, E, live, dtype, H):
    rng = np.random.default_rng(T * 1000 + H)
    slot_pos, _ = plan(rng, T, k, E, live)
    R = T * k + 3
    x = torch.randint(-100, 100, (T, H), dtype=torch.int64, device="cuda").to(dtype)
    sc = torch.randn((T, 5), device="cuda")
    out = torch.full((R, H), 77, device="cuda").to(dtype)
    out_sc = torch.full((R, 5), -7.0, device="cuda")
    want, want_sc = out.clone(), out_sc.clone()
    for t in range(T):
        for p in slot_pos[t]:
            if p >= 0:
                want[p], want_sc[p] = x[t], sc[t]
    mxmoe.moe_permute(x, dev(slot_pos), out, sc, out_sc)
    assert torch.equal(out, want) and torch.equal(out_sc, want_sc)
    alone = torch.full((R, H), 77, device="cuda").to(dtype)
    mxmoe.moe_permute(x, dev(slot_pos), alone)
    assert torch.equal(alone, want)


def test_permute_rows_that_lie_apart_and_positions_past_the_end():
    """A view of rows at an odd offset; places past out's rows are left out."""
    base = torch.randint(0, 255, (6, 100), dtype=torch.uint8, device="cuda")
    x = base[:, 3:53]
    pos = torch.tensor([[0, 9], [1, -5], [2, 2**31 - 1], [3, 4], [5, 6], [-1, 7]], dtype=torch.int32, device="cuda")
    out = torch.zeros((6, 50), dtype=torch.uint8, device="cuda")
    guard = torch.full((9, 50), 9, dtype=torch.uint8, device="cuda")
    guard[:6] = out
    mxmoe.moe_permute(x, pos, guard[:6])
    for p, t in ((0, 0), (1, 1), (2, 2), (3, 3), (4, 3), (5, 4)):
        assert torch.equal(guard[p], x[t])
    assert (guard[6:] == 9).all()
    one = base[2:3, 3:53]
    mxmoe.moe_permute(one, torch.tensor([[4]], dtype=torch.int32, device="cuda"), out)
    assert torch.equal(out[4], one[0])


def exact_back(o, w, slot_pos):
    T, k = slot_pos.shape
    y, most = np.zeros((T, o.shape[1])), np.zeros((T, o.shape[1]))
    for j in range(k):
        on = (slot_pos[:, j] >= 0) & (slot_pos[:, j] < len(o))
        v = (1.0 if w is None else w.astype(np.float64)[on, j, None]) * o[slot_pos[on, j]]
        y[on] += v
        most[on] += np.abs(v)
    return y, most


@pytest.mark.parametrize("T,k,E,live", CASES)
@pytest.mark.parametrize("o_type,y_type", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("H", [1, 7, 8, 9, 130, 2051])
def test_unpermute(T, k, E, live, o_type, y_type, H):
    rng = np.random.default_rng(H + T)
    slot_pos, _ = plan(rng, T, k, E, live)
    o, ov = typed(rng.standard_normal((T * k, H)), o_type)
    w = rng.random((T, k)).astype(np.float32)
    for weights in (w, None):
        y = torch.full((T, H), 7.0, device="cuda", dtype=y_type)
        mxmoe.moe_unpermute(o, None if weights is None else dev(weights), dev(slot_pos), y)
        want, most = exact_back(ov, weights, slot_pos)
        # k fp32 fmas, each off by half a step of a partial sum; then the result's own rounding
        tol = k * 2.0**-24 * most * (1 + 1e-6) + np.abs(want) * torch.finfo(y_type).eps / 2 * (1 + 1e-6)
        assert (np.abs(y.double().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("T,k,E,live", CASES)
@pytest.mark.parametrize("dy_type,o_type", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("H", [1, 7, 8, 65, 520, 2051])
def test_unpermute_grad(T, k, E, live, dy_type, o_type, H):
    rng = np.random.default_rng(H + T)
    slot_pos, _ = plan(rng, T, k, E, live)
    o, ov = typed(rng.standard_normal((T * k, H)), o_type)
    dy, dyv = typed(rng.standard_normal((T, H)), dy_type)
    w = rng.random((T, k)).astype(np.float32)
    d_o, dw = torch.full_like(o, 5.0), torch.full((T, k), 5.0, device="cuda")
    mxmoe.moe_unpermute_grad(dy, o, dev(w), dev(slot_pos), d_o, dw)
    want_o, want_w, most = torch.full_like(o, 5.0), np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j, p in enumerate(slot_pos[t]):
            if p >= 0:
                want_o[p] = (dy[t].float() * float(w[t, j])).to(o_type)     # one fp32 product, rounded once
                want_w[t, j], most[t, j] = dyv[t] @ ov[p], np.abs(dyv[t]) @ np.abs(ov[p])
    assert torch.equal(d_o, want_o)
    # a lane adds H / 64 products rounded up to eights and one, then six sums join the lanes
    tol = (-(-H // 512) * 8 + 7) * 2.0**-24 * most * (1 + 1e-5)
    assert (np.abs(dw.double().cpu().numpy() - want_w) <= tol).all()
    only_o, only_w = torch.full_like(o, 5.0), torch.full((T, k), 5.0, device="cuda")
    mxmoe.moe_unpermute_grad(dy, None, dev(w), dev(slot_pos), d_o=only_o)
    mxmoe.moe_unpermute_grad(dy, o, None, dev(slot_pos), dw=only_w)
    assert torch.equal(only_o, d_o) and torch.equal(only_w, dw)
    same = o.clone()                                                        # d_o in o's place
    mxmoe.moe_unpermute_grad(dy, same, dev(w), dev(slot_pos), same, only_w)
    named = torch.from_numpy(np.unique(slot_pos[slot_pos >= 0])).long().cuda()
    assert torch.equal(same[named], d_o[named]) and torch.equal(only_w, dw)


def test_the_gradient_of_unpermute_against_differences():
    """y is linear in o and in w: a difference quotient is the gradient, up to fp32's roundings of y."""
    rng = np.random.default_rng(3)
    T, k, H = 6, 3, 40
    slot_pos, _ = plan(rng, T, k, 8, 0.8)
    o, _ = typed(rng.integers(-4, 5, (T * k, H)), F32)
    dy, dyv = typed(rng.integers(-4, 5, (T, H)), F32)
    w = dev(rng.integers(1, 5, (T, k)).astype(np.float32))
    d_o, dw = torch.zeros_like(o), torch.zeros_like(w)
    mxmoe.moe_unpermute_grad(dy, o, w, dev(slot_pos), d_o, dw)

    def value(o, w):
        y = torch.zeros((T, H), device="cuda")
        mxmoe.moe_unpermute(o, w, dev(slot_pos), y)
        return float((y.double() * dy.double()).sum())

    at = value(o, w)                                                        # whole numbers: exact
    for t in range(T):
        for j in range(k):
            moved = w.clone()
            moved[t, j] += 1
            assert value(o, moved) - at == float(dw[t, j])
            if slot_pos[t, j] >= 0:
                p, h = int(slot_pos[t, j]), int(rng.integers(H))
                moved = o.clone()
                moved[p, h] += 1
                assert value(moved, w) - at == float(d_o[p, h])


def test_permute_and_back_are_each_other_s_gradient():
    """<permute(x), g> = <x, unpermute(g)> for whole numbers, exactly."""
    rng = np.random.default_rng(4)
    slot_pos, _ = plan(rng, 50, 4, 16, 0.7)
    x, xv = typed(rng.integers(-4, 5, (50, 77)), F32)
    g, gv = typed(rng.integers(-4, 5, (200, 77)), F32)
    out, y = torch.zeros_like(g), torch.zeros_like(x)
    mxmoe.moe_permute(x, dev(slot_pos), out)
    mxmoe.moe_unpermute(g, None, dev(slot_pos), y)
    assert float((out.double() * g.double()).sum()) == float((x.double() * y.double()).sum())


def test_special_values_stay_in_their_rows():
    """An infinity or NaN in a row of o reaches its own token only; one in a row that no slot names reaches none."""
    o = torch.ones((6, 70), device="cuda")
    o[1], o[5] = float("nan"), float("inf")
    pos = torch.tensor([[0, 2], [1, 3], [4, -1]], dtype=torch.int32, device="cuda")
    w = torch.ones((3, 2), device="cuda")
    y, dw = torch.zeros((3, 70), device="cuda"), torch.zeros((3, 2), device="cuda")
    mxmoe.moe_unpermute(o, w, pos, y)
    assert (y[0] == 2).all() and y[1].isnan().all() and (y[2] == 1).all()
    mxmoe.moe_unpermute_grad(torch.ones((3, 70), device="cuda"), o, w, pos, None, dw)
    assert dw[1, 0].isnan() and dw.nan_to_num(-1).tolist() == [[70, 70], [-1, 70], [70, 0]]
