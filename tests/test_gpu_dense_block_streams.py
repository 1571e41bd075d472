"""The dense block's helpers on a stream that they are given, with work of the current stream around them: bit for bit
the results of the same calls on the current stream."""
import numpy as np
import pytest
import torch

import dense_block_ref as ref
from block_scaled_fp8xfp4_amd.layer import AddNorm, DenseFFN, FP4Linear
from dense_block_ref import E2M1, E4M3, to_dev
from test_gpu_dense_block import typed

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.mark.parametrize("T", [1, 5, 300])
def test_helpers_on_a_given_stream(T):
    """norm -> projection and FFN -> norm on a side stream that is busy when the calls are made.  The residual's rows lie
    apart and are written on that stream only just before; the current stream writes over freed and new memory of the same
    sizes meanwhile."""
    H, I = 512, 288
    rng = np.random.default_rng(T)
    w, _ = typed(1 + 0.1 * rng.standard_normal(H), BF16)
    wp = [to_dev(t) for t in ref.weights(rng, H, H)]
    wf = [to_dev(t) for t in ref.weights(rng, 2 * I, H) + ref.weights(rng, H, I)]
    norm, proj, ffn = AddNorm(w, 1e-6), FP4Linear(*wp), DenseFFN(*wf, T, mid_fmt=E2M1)
    x, x2 = (typed(ref.activations(rng, T, H), BF16)[0] for _ in range(2))
    values, _ = typed(ref.activations(rng, T, H + 48), BF16)
    wide = torch.zeros_like(values)

    def block(residual, stream):
        h, q, sc, n = norm(x, residual[:, 16:16 + H], fmt=E4M3, hidden=True, stream=stream)
        y = proj(q, sc, E4M3, stream=stream)
        f = ffn(q, sc, E4M3, stream=stream)
        return (h, q, sc, n, y, f) + norm(f, h, x2=x2, fmt=E2M1, stream=stream)

    def clutter():
        for dtype, cols in ((BF16, H), (torch.uint8, H), (torch.uint8, H // 32), (torch.uint8, H // 2)):
            for _ in range(4):
                torch.empty((T, cols), dtype=dtype, device="cuda").fill_(3)

    want = block(values, None)
    torch.cuda.synchronize()
    side, load = torch.cuda.Stream(), torch.randn(2048, 2048, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    for k in range(3):
        with torch.cuda.stream(side):
            for _ in range(20):
                load = (load @ load).mul_(1e-2).clamp_(-1, 1)
            wide.copy_(values)
        got = block(wide, side.cuda_stream)
        clutter()
        side.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), k
        with torch.cuda.stream(side):
            wide.zero_()
        del got, a
        clutter()
    torch.cuda.synchronize()


def test_helpers_on_the_default_stream_by_its_handle():
    """0 is the default stream's handle, also where another stream is current."""
    H = 256
    rng = np.random.default_rng(1)
    w, _ = typed(1 + 0.1 * rng.standard_normal(H), BF16)
    x, r = (typed(ref.activations(rng, 4, H), BF16)[0] for _ in range(2))
    norm = AddNorm(w, 1e-6)
    want = norm(x, r, fmt=E2M1)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = norm(x, r, fmt=E2M1, stream=0)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_helper_captured_on_its_own_stream():
    """The stream that is being captured, by its handle: the graph replays on new rows."""
    H = 256
    rng = np.random.default_rng(2)
    proj = FP4Linear(*(to_dev(t) for t in ref.weights(rng, 64, H)))
    rows = [[to_dev(t) for t in ref.quantize(ref.activations(rng, 7, H), E4M3)] for _ in range(3)]
    want = [proj(*r, E4M3) for r in rows]
    a, a_sc = (t.clone() for t in rows[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = proj(a, a_sc, E4M3, stream=torch.cuda.current_stream().cuda_stream)
    for k in (1, 2, 0, 1):
        a.copy_(rows[k][0])
        a_sc.copy_(rows[k][1])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[k]), k
        assert torch.equal(proj(*rows[k], E4M3), want[k])
