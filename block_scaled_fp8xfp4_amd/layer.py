"""Device-side convenience wrapper around the C-ABI: uploads and quantizes a
MoE layer on the GPU (with the library's own quantizer kernel) and owns the
route / FFN workspaces.  Every computation is a libmxmoe.so call."""
import contextlib

import numpy as np
import torch

from . import mxmoe


def _dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)) if isinstance(a, np.ndarray) else a
    return t.to("cuda", dtype=dtype) if dtype is not None else t.to("cuda")


def quantize(v, fmt):
    """fp32/bf16 device tensor [..., cols] -> (codes, scales) device uint8 tensors."""
    cols = v.shape[-1]
    rows = v.numel() // cols
    qcols = cols if fmt == mxmoe.MX_FMT_E4M3 else cols // 2
    q = torch.empty(v.shape[:-1] + (qcols,), dtype=torch.uint8, device=v.device)
    sc = torch.empty(v.shape[:-1] + (cols // 32,), dtype=torch.uint8, device=v.device)
    if rows:
        mxmoe.mx_quantize(v.contiguous(), q, sc, fmt)
    return q, sc


def quantize_experts(w_host, chunk=16):
    """fp32 host weights [E, R, C] -> packed E2M1 [E, R, C/2] + E8M0 [E, R, C/32] on the GPU."""
    E, R, C = w_host.shape
    q = torch.empty((E, R, C // 2), dtype=torch.uint8, device="cuda")
    sc = torch.empty((E, R, C // 32), dtype=torch.uint8, device="cuda")
    for e0 in range(0, E, chunk):
        e1 = min(E, e0 + chunk)
        src = _dev(w_host[e0:e1])
        mxmoe.mx_quantize(src, q[e0:e1], sc[e0:e1], mxmoe.MX_FMT_E2M1)
    torch.cuda.synchronize()
    return q, sc


class RouterLogits:
    """Owns the workspace of moe_router_logits for up to T rows."""

    def __init__(self, T, H, E):
        self.T, self.H, self.E = T, H, E
        n = max(mxmoe.moe_router_logits_workspace_bytes(t, H, E) for t in range(1, min(T, 1024) + 1))
        self.ws = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")

    def __call__(self, hidden, w_gate, logits, stream=None):
        if hidden.shape[0] > self.T:
            raise ValueError("RouterLogits: more rows than sized for")
        mxmoe.moe_router_logits(hidden, w_gate, logits, self.ws, stream)
        return logits


class Route:
    def __init__(self, T, E, k):
        dev = "cuda"
        self.T, self.E, self.k = T, E, k
        self.ids = torch.empty((T, k), dtype=torch.int32, device=dev)
        self.w = torch.empty((T, k), dtype=torch.float32, device=dev)
        self.offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
        self.perm = torch.empty(T * k, dtype=torch.int32, device=dev)
        self.slot_pos = torch.empty((T, k), dtype=torch.int32, device=dev)
        self.ws = torch.empty(mxmoe.moe_route_workspace_bytes(T, E, k), dtype=torch.uint8, device=dev)

    def __call__(self, logits, survival=None, skip_below=0.2, stream=None, anchor=None):
        """Skip mode, or router-live mode when anchor (int32 [T]) is given
        (then skip_below is the reuse threshold)."""
        if anchor is None:
            mxmoe.moe_route(logits, self.k, survival, skip_below, self.ids, self.w, self.offsets, self.perm,
                            self.slot_pos, self.ws, stream)
        else:
            mxmoe.moe_route_live(logits, self.k, survival, skip_below, anchor, self.ids, self.w, self.offsets,
                                 self.perm, self.slot_pos, self.ws, stream)
        return self


class ExpertFFN:
    def __init__(self, T, H, E, I, k):
        self.T, self.H, self.E, self.I, self.k = T, H, E, I, k
        self.ws = torch.empty(mxmoe.moe_expert_ffn_workspace_bytes(T, H, E, I, k), dtype=torch.uint8, device="cuda")
        self.y = torch.empty((T, H), dtype=torch.float32, device="cuda")

    def __call__(self, x, x_sc, route, w13, w13_sc, w2, w2_sc, stream=None):
        mxmoe.moe_expert_ffn(x, x_sc, route.w, route.offsets, route.perm, route.slot_pos, self.k, w13, w13_sc,
                             w2, w2_sc, self.E, self.I, self.y, self.ws, stream)
        return self.y

    def ws_views(self):
        """Workspace regions as tensors: q [T*k, I], q_sc [T*k, I/32] (uint8)
        and o [T*k, H] (fp32, T > 1)."""
        Tk, H, I = self.T * self.k, self.H, self.I
        oq, oqs, oo = mxmoe.moe_ws_layout(self.T, H, I, self.k)
        q = self.ws[oq:oq + Tk * I].view(Tk, I)
        sc = self.ws[oqs:oqs + Tk * (I // 32)].view(Tk, I // 32)
        o = self.ws[oo:oo + Tk * H * 4].view(torch.float32).view(Tk, H)
        return q, sc, o


def _under(stream):
    """The context of a helper that makes tensors and launches on stream (a raw handle; None: torch's current stream, 0: the
    default one).  What it makes then belongs to that stream, as under torch.cuda.stream: memory that the allocator hands
    out or takes back is not in use by work elsewhere, and a copy is ordered before the kernel that reads it."""
    if stream is None:
        return contextlib.nullcontext()
    d = torch.cuda.current_device()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream, device=d) if stream else torch.cuda.default_stream(d))


class AddNorm:
    """Residual addition + root-mean-square norm (mx_add_rmsnorm) with a weight [H].  A residual whose rows lie apart is
    copied first, since h shares its layout."""

    def __init__(self, weight, eps=1e-6):
        self.weight, self.eps = weight, eps

    def __call__(self, x, residual=None, x2=None, fmt=None, hidden=False, stream=None):
        """(h, ...) with the codes and scales of the normed rows when fmt is given, then with the rows themselves in
        bf16 when hidden is set.  h is the new residual stream, in the residual's type (x's without one)."""
        T, H = x.shape
        with _under(stream):
            h = torch.empty((T, H), dtype=x.dtype if residual is None else residual.dtype, device=x.device)
            if residual is not None and T > 1 and residual.stride(0) != H:
                residual = residual.contiguous()
            out, q, sc, n = [h], None, None, None
            if fmt is not None:
                q = torch.empty((T, H if fmt == mxmoe.MX_FMT_E4M3 else H // 2), dtype=torch.uint8, device=x.device)
                sc = torch.empty((T, H // 32), dtype=torch.uint8, device=x.device)
                out += [q, sc]
            if hidden:
                n = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
                out.append(n)
            mxmoe.mx_add_rmsnorm(x, self.weight, self.eps, residual, x2, h, n, q, sc,
                                 mxmoe.MX_FMT_E4M3 if fmt is None else fmt, stream)
        return tuple(out)


class FP4Linear:
    """A dense projection with MXFP4 weights [N, K/2] + scales [N, K/32] (fp4_block_gemm)."""

    def __init__(self, w, w_sc):
        self.w, self.w_sc = w, w_sc

    def __call__(self, a, a_sc, a_fmt, dtype=torch.bfloat16, stream=None):
        with _under(stream):
            y = torch.empty((a.shape[0], self.w.shape[0]), dtype=dtype, device=a.device)
            mxmoe.fp4_block_gemm(a, a_sc, a_fmt, self.w, self.w_sc, y, stream)
        return y


class DenseFFN:
    """A dense SwiGLU FFN with MXFP4 weights (fp4_dense_ffn); owns the workspace of up to T rows, which its calls and the
    graphs captured of them share: they must not overlap, and a call on another stream than the one that made the object
    comes after that stream's work, the object's end after the call's."""

    def __init__(self, w13, w13_sc, w2, w2_sc, T, mid_fmt=mxmoe.MX_FMT_E4M3):
        self.weights, self.T, self.mid_fmt = (w13, w13_sc, w2, w2_sc), T, mid_fmt
        self.H, self.I = w2.shape[0], w2.shape[1] * 2
        n = max(mxmoe.fp4_dense_ffn_workspace_bytes(t, self.H, self.I, mid_fmt) for t in (1, T))
        self.ws = torch.empty(max(n, 256), dtype=torch.uint8, device=w13.device)

    def __call__(self, x, x_sc, x_fmt, dtype=torch.bfloat16, stream=None):
        if x.shape[0] > self.T:
            raise ValueError("DenseFFN: more rows than sized for")
        with _under(stream):
            y = torch.empty((x.shape[0], self.H), dtype=dtype, device=x.device)
            mxmoe.fp4_dense_ffn(x, x_sc, x_fmt, *self.weights, self.mid_fmt, y, self.ws, stream)
        return y
