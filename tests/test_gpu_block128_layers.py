"""The experts' tokens, casts and products together, as layers use them: the FFN of FP8 experts, projections with their
gradients, on streams and in captured graphs."""
import numpy as np
import pytest
import torch

import block128_ref as ref
from block128_ref import BF16, F32, B, blocks, dev, typed
from block_scaled_fp8xfp4_amd import mxmoe
from block_scaled_fp8xfp4_amd.layer import (ExpertFFN128, ExpertLinear128, FP8Linear128, Route, quantize128, quantize128_t)

pytestmark = pytest.mark.gpu


def experts(rng, E, N, K, size):
    w, sc = zip(*[ref.cast(rng.standard_normal((N, K)) * size, B, B) for _ in range(E)])
    return np.stack(w), np.stack(sc)


def ffn_weights(rng, E, H, I):
    return experts(rng, E, 2 * I, H, H ** -0.5), experts(rng, E, H, I, I ** -0.5)


@pytest.mark.parametrize("T,k,E,H,I,skip", [(1, 2, 8, 256, 128, False), (5, 3, 7, 272, 144, True), (40, 4, 16, 400, 208, True),
                                            (300, 2, 4, 256, 320, False)])
def test_expert_ffn(T, k, E, H, I, skip):
    """Route, cast, sort, products and back against 64 bits, step by step: a gate/up value that falls on the other side of a
    bf16 border is off by 2^-8, and where it is its block's largest, or its quotient lies near a border between codes, codes
    move by a step of 2^-4 to 2^-3.  With values 3e-5 of the norm off, 1 in 200 crosses; then 1 in 16 moves its code (error^2
    2 / 200 / 16 * 0.087^2 = 5e-6 of the norm^2) and 1 block in 100 has another scale (as much again): 3e-3 of the norm is the
    usual error, one row's several times that, so the codes are made from the kernel's own gate/up values, which are compared
    themselves.  Matrix cores cut 2^-10 of the sum of magnitudes at most, bf16 rounds by 2^-8 at most."""
    rng = np.random.default_rng(T)
    (w13, s13), (w2, s2) = ffn_weights(rng, E, H, I)
    x, xv = typed(rng.standard_normal((T, H)), BF16)
    route = Route(T, E, k)
    surv = torch.rand(T, device="cuda") if skip else None
    route(torch.randn((T, E), device="cuda"), surv, 0.3)
    y = ExpertFFN128(*[dev(v) for v in (w13, s13, w2, s2)])(x, route)
    xq, x_sc = quantize128(x)
    xs, xs_sc = torch.zeros((T * k, H), dtype=torch.uint8, device="cuda"), torch.ones((T * k, blocks(H)), device="cuda")
    mxmoe.moe_permute(xq, route.slot_pos, xs, x_sc, xs_sc)
    gu_kept = torch.zeros((T * k, 2 * I), dtype=BF16, device="cuda")
    mxmoe.fp8_block128_grouped_gemm(xs, xs_sc, dev(w13), dev(s13), route.offsets, gu_kept)
    gu_kept = gu_kept.double().cpu().numpy()

    def product(v, w):
        exact, cut = v @ w.T, 2.0**-10 * (np.abs(v) @ np.abs(w).T)
        return exact, cut + 2.0**-8 * (np.abs(exact) + cut)

    q, sc = ref.cast(xv, 1, B)
    rows = ref.wide(q, sc, 1)
    want, most = np.zeros((T, H)), np.zeros((T, H))
    ids, w, pos = route.ids.cpu().numpy(), route.w.double().cpu().numpy(), route.slot_pos.cpu().numpy()
    for t in range(T):
        for j in range(k):
            if pos[t, j] < 0:
                continue
            e = ids[t, j]
            exact, off = product(rows[t], ref.wide(w13[e], s13[e], B))
            gu = gu_kept[pos[t, j]]
            assert (np.abs(gu - exact) <= off).all()
            a = (gu[:I] / (1 + np.exp(-gu[:I])) * gu[I:]).astype(np.float32).astype(np.float64)
            aq, a_sc = ref.cast(a[None], 1, B)
            o, off = product(ref.wide(aq, a_sc, 1)[0], ref.wide(w2[e], s2[e], B))
            want[t] += w[t, j] * o
            most[t] += w[t, j] * (off + k * 2.0**-23 * (np.abs(o) + off))      # and fp32 sums over the slots
    got = y.double().cpu().numpy()
    dead = (pos < 0).all(1)
    assert (got[dead] == 0).all() and dead.any() <= skip
    assert (np.abs(got - want) <= most).all()
    assert np.linalg.norm(got - want) <= 2.0**-8 * np.linalg.norm(want)                # a bf16 result's rounding, and little more


def test_a_token_s_output_does_not_depend_on_the_others():
    rng = np.random.default_rng(2)
    T, k, E, H, I = 200, 3, 8, 256, 144
    (w13, s13), (w2, s2) = ffn_weights(rng, E, H, I)
    ffn = ExpertFFN128(*[dev(v) for v in (w13, s13, w2, s2)])
    x, logits = torch.randn((T, H), device="cuda").to(BF16), torch.randn((T, E), device="cuda")
    full = ffn(x, Route(T, E, k)(logits))
    for rows in ([0], [199], list(range(50, 67)), list(range(0, 200, 3))):
        at = torch.tensor(rows, device="cuda")
        y = ffn(x[at].contiguous(), Route(len(rows), E, k)(logits[at].contiguous()))
        assert torch.equal(y, full[at])


def sevens(rng, rows, cols, cut=None):
    """Whole numbers -7 .. 7 with a 7 in every block of any direction: casts of them are exact."""
    v = rng.integers(-7, 8, (rows, cols)).astype(np.float64)
    for r0 in range(0, rows, 16):
        v[r0:r0 + 16][np.arange(min(16, rows - r0)), rng.integers(0, min(cols, 16), min(16, rows - r0))] = 7
    v[:, ::16] = 7
    v[::16] = 7
    if cut:
        v[[c for c in cut if c < rows]] = 7
    return v


@pytest.mark.parametrize("T,N,K", [(1, 16, 16), (130, 144, 272), (300, 400, 160)])
def test_linear_and_its_gradients(T, N, K):
    """Exact for whole numbers: the gradients are their formulas, and the differences of the layer's own results."""
    rng = np.random.default_rng(T)
    (x, xv), (g, gv), wv = typed(sevens(rng, T, K), BF16), typed(sevens(rng, T, N), BF16), sevens(rng, N, K)
    layer = FP8Linear128(*quantize128(dev(wv.astype(np.float32)), 128), train=True)
    y = layer(x, dtype=F32)
    assert np.array_equal(y.double().cpu().numpy(), xv @ wv.T)
    assert np.array_equal(layer.input_grad(g, dtype=F32).double().cpu().numpy(), gv @ wv)
    dw = layer.weight_grad(g, x).double().cpu().numpy()
    assert np.array_equal(dw, gv.T @ xv)
    for _ in range(5):
        n, k = rng.integers(N), rng.integers(K)
        step = 1 if wv[n, k] < 7 else -1
        moved = wv.copy()
        moved[n, k] += step
        if moved.reshape(-1)[0] != 7 or not (np.abs(moved[:128, :128]).max() == 7):
            continue
        q, sc = quantize128(dev(moved.astype(np.float32)), 128)
        diff = FP8Linear128(q, sc)(x, dtype=F32).double() - y.double()
        assert float((diff * g.double()).sum()) == step * dw[n, k]
    with pytest.raises(ValueError):
        FP8Linear128(layer.w, layer.w_sc).input_grad(g)


@pytest.mark.parametrize("bounds,N,K", [([0, 1], 16, 32), ([0, 0, 5, 5, 133, 400, 400], 144, 96), ([0, 200, 330], 48, 272)])
def test_expert_linear_and_its_gradients(bounds, N, K):
    rng = np.random.default_rng(N)
    E, R = len(bounds) - 1, bounds[-1]
    starts = [b + 128 * i for a, b in zip(bounds, bounds) for i in range(4)]
    (x, xv), (g, gv) = typed(sevens(rng, R, K, starts), BF16), typed(sevens(rng, R, N, starts), BF16)
    wv = np.stack([sevens(rng, N, K) for _ in range(E)])
    off = dev(np.array(bounds, np.int32))
    layer = ExpertLinear128(*quantize128(dev(wv.astype(np.float32)), 128), train=True)
    y, dx, dw = layer(x, off, dtype=F32), layer.input_grad(g, off, dtype=F32), layer.weight_grad(g, x, off)
    for e, (i, j) in enumerate(zip(bounds, bounds[1:])):
        assert np.array_equal(y[i:j].double().cpu().numpy(), xv[i:j] @ wv[e].T)
        assert np.array_equal(dx[i:j].double().cpu().numpy(), gv[i:j] @ wv[e])
        assert np.array_equal(dw[e].double().cpu().numpy(), gv[i:j].T @ xv[i:j])


def test_training_step_of_routed_experts():
    """Sort, product, back, and all of their gradients, against the formulas on the cast values in 64 bits: matrix cores cut
    2^-10 of the sum of magnitudes at most, fp32 rounds once per block and scale, bf16 rows once."""
    rng = np.random.default_rng(5)
    T, k, E, H, N = 150, 2, 6, 272, 144
    x, xv = typed(rng.standard_normal((T, H)), BF16)
    dy, dyv = typed(rng.standard_normal((T, N)), BF16)
    w, w_sc = experts(rng, E, N, H, 0.05)
    layer = ExpertLinear128(dev(w), dev(w_sc), train=True)
    route = Route(T, E, k)(torch.randn((T, E), device="cuda"))
    R = T * k
    xs = torch.empty((R, H), dtype=BF16, device="cuda")
    mxmoe.moe_permute(x, route.slot_pos, xs)
    o = layer(xs, route.offsets, dtype=BF16)
    y = torch.empty((T, N), device="cuda")
    mxmoe.moe_unpermute(o, route.w, route.slot_pos, y)
    d_o, dwr = torch.empty_like(o), torch.empty_like(route.w)
    mxmoe.moe_unpermute_grad(dy, o, route.w, route.slot_pos, d_o, dwr)
    dxs = layer.input_grad(d_o, route.offsets, dtype=F32)
    dx = torch.empty((T, H), device="cuda")
    mxmoe.moe_unpermute(dxs, None, route.slot_pos, dx)
    dw = layer.weight_grad(d_o, xs, route.offsets)
    host = lambda t: t.double().cpu().numpy()  # noqa: E731
    pos, off, wr = route.slot_pos.cpu().numpy(), route.offsets.cpu().numpy(), host(route.w)
    d_ov = host(d_o)
    for t in range(T):
        for j in range(k):
            assert np.array_equal(d_ov[pos[t, j]], ref.bf16(np.float32(wr[t, j]) * dyv[t].astype(np.float32)))
    rows = np.empty((R, H))
    rows[pos] = xv[:, None]
    want_dx = np.zeros((T, H))
    for e in range(E):
        i, j = off[e], off[e + 1]
        if i == j:
            continue
        wv = ref.wide(w[e], w_sc[e], B)
        g, x_ = ref.wide(*ref.cast(d_ov[i:j], 1, B), 1), ref.wide(*ref.cast(rows[i:j], 1, B), 1)
        slack = lambda most, n: (2.0**-10 + (blocks(n) + 2) * 2.0**-23) * most  # noqa: E731
        want = x_ @ wv.T
        tol = slack(np.abs(x_) @ np.abs(wv).T, H) * (1 + 2.0**-8) + np.abs(want) * 2.0**-8
        assert (np.abs(host(o)[i:j] - want) <= tol).all()
        assert (np.abs(host(dxs)[i:j] - g @ wv) <= slack(np.abs(g) @ np.abs(wv), N)).all()
        gc, xc = [ref.wide(*ref.cast(v[i:j].T, 1, B), 1) for v in (d_ov, rows)]
        assert (np.abs(host(dw)[e] - gc @ xc.T) <= slack(np.abs(gc) @ np.abs(xc).T, j - i)).all()
    dxv = host(dxs)
    want_dx, most = dxv[pos].sum(1), np.abs(dxv[pos]).sum(1)
    assert (np.abs(host(dx) - want_dx) <= k * 2.0**-24 * most).all()
    ov = host(o)
    most = (np.abs(dyv)[:, None] * np.abs(ov[pos])).sum(-1)
    assert (np.abs(host(dwr) - (dyv[:, None] * ov[pos]).sum(-1)) <= 20 * 2.0**-24 * most).all()


def test_layers_on_a_given_stream():
    """Bit for bit the results of the current stream, with that stream busy and the current one writing over memory."""
    rng = np.random.default_rng(6)
    T, k, E, H, I = 60, 2, 6, 256, 128
    (w13, s13), (w2, s2) = ffn_weights(rng, E, H, I)
    ffn = ExpertFFN128(*[dev(v) for v in (w13, s13, w2, s2)])
    w, w_sc = experts(rng, E, H, H, 0.1)
    lin, dense = ExpertLinear128(dev(w), dev(w_sc), train=True), FP8Linear128(dev(w[0]), dev(w_sc[0]), train=True)
    route = Route(T, E, k)(torch.randn((T, E), device="cuda"))
    values = torch.randn((T, H), device="cuda").to(BF16)
    rows = torch.randn((T * k, H), device="cuda").to(BF16)
    x = torch.zeros_like(values)

    def block(x, stream):
        y = ffn(x, route, dtype=BF16, stream=stream)
        z = lin(rows, route.offsets, stream=stream)
        return (y, z, lin.input_grad(z, route.offsets, stream=stream), lin.weight_grad(z, rows, route.offsets, stream=stream),
                dense(y, stream=stream), dense.input_grad(x, stream=stream), dense.weight_grad(y, x, stream=stream))

    want = block(values, None)
    torch.cuda.synchronize()
    side, load = torch.cuda.Stream(), torch.randn(2048, 2048, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(side):
            for _ in range(20):
                load = (load @ load).mul_(1e-2).clamp_(-1, 1)
            x.copy_(values)
        got = block(x, side.cuda_stream)
        for shape in ((T, H), (T * k, H), (T * k, 2 * I), (E, H, H)):
            torch.empty(shape, dtype=BF16, device="cuda").fill_(3)
        side.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        with torch.cuda.stream(side):
            x.zero_()
        del got, a


def test_layers_in_two_graphs():
    """Two captures of the same layers, replayed several times in turns with new inputs and eager work between."""
    rng = np.random.default_rng(7)
    T, k, E, H, I = 48, 2, 8, 256, 144
    (w13, s13), (w2, s2) = ffn_weights(rng, E, H, I)
    ffn = ExpertFFN128(*[dev(v) for v in (w13, s13, w2, s2)])
    w, w_sc = experts(rng, E, 2 * I, H, 0.1)
    lin = ExpertLinear128(dev(w), dev(w_sc), train=True)
    cases = []
    for _ in range(2):
        x, logits, route = torch.zeros((T, H), device="cuda", dtype=BF16), torch.zeros((T, E), device="cuda"), Route(T, E, k)
        rows = torch.zeros((T * k, H), device="cuda", dtype=BF16)

        def work(x=x, logits=logits, route=route, rows=rows):
            route(logits)
            y = ffn(x, route)
            mxmoe.moe_permute(x, route.slot_pos, rows)
            z = lin(rows, route.offsets)
            dw = torch.empty_like(route.w)
            mxmoe.moe_unpermute_grad(torch.ones((T, 2 * I), device="cuda"), z, route.w, route.slot_pos, None, dw)
            return y, z, lin.input_grad(z, route.offsets), lin.weight_grad(z, rows, route.offsets), dw
        x.normal_()
        logits.normal_()
        work()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = work()
        cases.append((x, logits, work, graph, out))
    for i in range(6):
        x, logits, work, graph, out = cases[i % 2]
        x.normal_()
        logits.normal_()
        graph.replay()
        got = [t.clone() for t in out]
        want = work()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), i


def test_the_same_bits_again():
    rng = np.random.default_rng(8)
    a, a_sc, w, w_sc = [dev(v) for v in ref.cast(rng.standard_normal((5000, 1024)), 1, B) + ref.cast(rng.standard_normal((1500, 1024)), B, B)]
    y = [torch.empty((5000, 1500), device="cuda") for _ in range(3)]
    for t in y:
        mxmoe.fp8_block128_gemm(a, a_sc, w, w_sc, t)
    assert torch.equal(y[0], y[1]) and torch.equal(y[0], y[2])
    q = [quantize128_t(y[0].to(BF16)) for _ in range(2)]
    assert torch.equal(q[0][0], q[1][0]) and torch.equal(q[0][1], q[1][1])
