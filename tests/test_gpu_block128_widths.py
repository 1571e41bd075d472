"""The gradients of layers of any number of outputs: a projection takes any N, so its input gradient does, whose sum runs over
N and whose cast needs whole 16s."""
import numpy as np
import pytest
import torch

from block128_ref import BF16, F32, dev, typed
from block_scaled_fp8xfp4_amd.layer import ExpertLinear128, FP8Linear128, quantize128
from test_gpu_block128_layers import sevens

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,N,K", [(3, 1, 16), (5, 17, 144), (130, 130, 272), (40, 250, 32), (300, 1001, 160)])
def test_linear_gradients_of_any_number_of_outputs(T, N, K):
    """Exact for whole numbers."""
    rng = np.random.default_rng(N)
    (x, xv), wv = typed(sevens(rng, T, K), BF16), sevens(rng, N, K)
    layer = FP8Linear128(*quantize128(dev(wv.astype(np.float32)), 128), train=True)
    assert np.array_equal(layer(x, dtype=F32).double().cpu().numpy(), xv @ wv.T)
    for dtype in (BF16, F32):
        g, gv = typed(sevens(rng, T, N), dtype)
        assert np.array_equal(layer.input_grad(g, dtype=F32).double().cpu().numpy(), gv @ wv)
        assert np.array_equal(layer.weight_grad(g, x).double().cpu().numpy(), gv.T @ xv)
        wide = torch.full((T, N + 5), 9, dtype=dtype, device="cuda")
        wide[:, 2:2 + N] = g
        if N % 16:                                          # copied with its zeros, so it may lie anywhere
            assert torch.equal(layer.input_grad(wide[:, 2:2 + N], dtype=F32), layer.input_grad(g, dtype=F32))
    with pytest.raises(ValueError):
        layer.input_grad(torch.ones((T, -(-N // 16) * 16 + (N % 16 == 0)), device="cuda"))


@pytest.mark.parametrize("bounds,N,K", [([0, 1], 1, 32), ([0, 0, 5, 5, 133, 400, 400], 130, 96), ([0, 200, 330], 50, 272)])
def test_expert_linear_gradients_of_any_number_of_outputs(bounds, N, K):
    rng = np.random.default_rng(N)
    E, R = len(bounds) - 1, bounds[-1]
    starts = [b + 128 * i for b in bounds for i in range(4)]
    (x, xv), (g, gv) = typed(sevens(rng, R, K, starts), BF16), typed(sevens(rng, R, N, starts), BF16)
    wv = np.stack([sevens(rng, N, K) for _ in range(E)])
    off = dev(np.array(bounds, np.int32))
    layer = ExpertLinear128(*quantize128(dev(wv.astype(np.float32)), 128), train=True)
    y, dx, dw = layer(x, off, dtype=F32), layer.input_grad(g, off, dtype=F32), layer.weight_grad(g, x, off)
    for e, (i, j) in enumerate(zip(bounds, bounds[1:])):
        assert np.array_equal(y[i:j].double().cpu().numpy(), xv[i:j] @ wv[e].T)
        assert np.array_equal(dx[i:j].double().cpu().numpy(), gv[i:j] @ wv[e])
        assert np.array_equal(dw[e].double().cpu().numpy(), gv[i:j].T @ xv[i:j])
    with pytest.raises(ValueError):
        layer.input_grad(torch.ones((R, -(-N // 16) * 16), device="cuda"), off)


def test_input_gradient_in_a_graph():
    """The copy with zeros is captured too, and read anew at every replay."""
    T, N, K = 20, 75, 64
    layer = FP8Linear128(*quantize128(torch.randn((N, K), device="cuda"), 128), train=True)
    g = torch.randn((T, N), device="cuda").to(BF16)
    layer.input_grad(g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.input_grad(g)
    for _ in range(4):
        g.normal_()
        graph.replay()
        got = out.clone()
        assert torch.equal(got, layer.input_grad(g))
        torch.cuda.synchronize()
