"""The dense block's helpers when they are given a stream, without a GPU: every tensor that a call makes itself (outputs, a
copy of a residual whose rows lie apart) is allocated and written under that stream, and the entry point is called with
it.  Made on the current stream instead, a copy is not ordered before the kernel that reads it, and a block that the
allocator hands out or takes back there may still be in use."""
import contextlib

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from block_scaled_fp8xfp4_amd import layer, mxmoe
from block_scaled_fp8xfp4_amd.layer import AddNorm, DenseFFN, FP4Linear

HANDLE, DEFAULT = 0x5150, "the default stream"


class Made(TorchDispatchMode):
    """Notes for every operation that makes a tensor under which stream it ran."""

    def __init__(self, current):
        super().__init__()
        self.current, self.seen = current, []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        if any(s in func.__name__ for s in ("empty", "clone", "copy", "contiguous")):
            self.seen.append((func.__name__, self.current[-1]))
        return func(*args, **(kwargs or {}))


@pytest.fixture
def streams(monkeypatch):
    """The stack of current streams, with torch.cuda's contexts replaced by ones that push to it."""
    current = [None]

    @contextlib.contextmanager
    def under(stream):
        current.append(stream)
        yield
        current.pop()

    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None, **kw: handle)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: DEFAULT)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return current


def calls(monkeypatch, name):
    made = []
    monkeypatch.setattr(mxmoe, name, lambda *a, **k: made.append((a, k)))
    return made


def u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


@pytest.mark.parametrize("handle,where", [(HANDLE, HANDLE), (0, DEFAULT), (None, None)])
def test_helpers_allocate_under_the_given_stream(monkeypatch, streams, handle, where):
    norm_calls, gemm_calls, ffn_calls = (calls(monkeypatch, n) for n in ("mx_add_rmsnorm", "fp4_block_gemm", "fp4_dense_ffn"))
    monkeypatch.setattr(mxmoe, "fp4_dense_ffn_workspace_bytes", lambda *a: 1024)
    x, wide = torch.zeros(3, 64), torch.arange(3 * 96.0).view(3, 96)
    norm, linear = AddNorm(torch.ones(64)), FP4Linear(u8(8, 32), u8(8, 2))
    ffn = DenseFFN(u8(64, 32), u8(64, 2), u8(64, 16), u8(64, 1), 3)
    with Made(streams) as made:
        out = norm(x, wide[:, 16:80], fmt=mxmoe.MX_FMT_E4M3, hidden=True, stream=handle)
        y = linear(u8(3, 64), u8(3, 2), mxmoe.MX_FMT_E4M3, stream=handle)
        z = ffn(u8(3, 64), u8(3, 2), mxmoe.MX_FMT_E4M3, stream=handle)
    assert len(made.seen) >= 6 and {s for _, s in made.seen} == {where}, made.seen
    assert len(out) == 4 and out[0].shape == (3, 64) and y.shape == (3, 8) and z.shape == (3, 64)
    for (args, kwargs), at in ((norm_calls[0], 10), (gemm_calls[0], 6), (ffn_calls[0], 10)):
        assert (args[at] if len(args) > at else kwargs["stream"]) == handle
    args = norm_calls[0][0]
    assert torch.equal(args[3], wide[:, 16:80])
    assert streams == [None]


def test_a_residual_of_whole_rows_is_not_copied(monkeypatch, streams):
    made = calls(monkeypatch, "mx_add_rmsnorm")
    r = torch.zeros(3, 64)
    AddNorm(torch.ones(64))(torch.zeros(3, 64), r, stream=HANDLE)
    assert made[0][0][3] is r
    one = torch.zeros(3, 96)[1:2, :64]
    AddNorm(torch.ones(64))(torch.zeros(1, 64), one, stream=HANDLE)
    assert made[1][0][3] is one
