"""Thin ctypes binding of libmxmoe.so (include/mxmoe.h).

Argument marshalling only: torch tensors supply device memory and the current
HIP stream; every step of the computation runs in the library's kernels.  The
binding raises if the library is missing, never falls back to another path.
"""
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmxmoe.so")

MX_OK, MX_EINVAL, MX_EUNSUPPORTED, MX_EWORKSPACE, MX_EHIP = 0, -1, -2, -3, -4
MX_FMT_E4M3, MX_FMT_E2M1 = 0, 1
MX_IN_F32, MX_IN_BF16 = 0, 1
MX_OUT_BF16, MX_OUT_F32 = 0, 1

# every entry point declared in include/mxmoe.h
EXPORTS = ("mx_quantize", "moe_router_logits_workspace_bytes", "moe_router_logits", "moe_route_workspace_bytes", "moe_route", "moe_route_live", "moe_expert_ffn_workspace_bytes",
           "moe_ws_layout", "moe_expert_ffn", "fp8_block_gemm", "mx_status_string",
           "mx_last_variant", "mx_set_ffn_path", "mx_set_layer1_single_launch", "mx_check_requant", "mx_set_phase_events",
           "moe_shared_expert_workspace_bytes", "moe_shared_expert", "mx_prefetch",
           "moe_layer_decode1", "mx_set_ffn_diag", "moe_expert_ffn_noalloc", "moe_expert_ffn_noalloc_max_bytes",
           "moe_layer_decode1_shared_workspace_bytes", "moe_layer_decode1_shared",
           "mx_dequantize", "mx_swiglu_quantize", "mx_add_rmsnorm", "fp4_block_gemm",
           "fp4_dense_ffn_workspace_bytes", "fp4_dense_ffn",
           "moe_permute", "moe_unpermute", "moe_unpermute_grad",
           "fp8_quantize128", "fp8_swiglu_quantize128", "fp8_quantize128_t_cols", "fp8_quantize128_t",
           "fp8_block128_gemm", "fp8_block128_grouped_gemm", "fp8_block128_grouped_wgrad")

_lib = None


class MXError(RuntimeError):
    def __init__(self, status, name):
        self.status = status
        super().__init__(f"{name}: {status_string(status)} ({status})")


def load():
    """Load libmxmoe.so (built by block_scaled_fp8xfp4_amd.build); raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run `python -m block_scaled_fp8xfp4_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, SZ, F32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    lib.mx_quantize.restype = I32
    lib.mx_quantize.argtypes = [P, I32, I64, I64, I32, P, P, P]
    lib.moe_router_logits.restype = I32
    lib.moe_router_logits.argtypes = [P, I32, I32, P, I32, P, P, SZ, P]
    lib.moe_router_logits_workspace_bytes.restype = SZ
    lib.moe_router_logits_workspace_bytes.argtypes = [I32, I32, I32]
    lib.moe_route_workspace_bytes.restype = SZ
    lib.moe_route_workspace_bytes.argtypes = [I32, I32, I32]
    lib.moe_route.restype = I32
    lib.moe_route.argtypes = [P, I32, I32, I32, P, F32, P, P, P, P, P, P, SZ, P]
    lib.moe_route_live.restype = I32
    lib.moe_route_live.argtypes = [P, I32, I32, I32, P, F32, P, P, P, P, P, P, P, SZ, P]
    lib.moe_expert_ffn_workspace_bytes.restype = SZ
    lib.moe_expert_ffn_workspace_bytes.argtypes = [I32, I32, I32, I32, I32]
    lib.moe_ws_layout.restype = I32
    lib.moe_ws_layout.argtypes = [I32, I32, I32, I32, P, P, P]
    lib.mx_set_ffn_diag.restype = I32
    lib.mx_set_ffn_diag.argtypes = [P, SZ]
    lib.moe_expert_ffn.restype = I32
    lib.moe_expert_ffn.argtypes = [P, P, I32, I32, P, P, P, P, I32, P, P, P, P, I32, I32, P, P, SZ, P]
    lib.moe_expert_ffn_noalloc.restype = I32
    lib.moe_expert_ffn_noalloc.argtypes = [P, P, I32, I32, P, P, P, P, I32, P, P, P, P, I32, I32, P, P]
    lib.moe_expert_ffn_noalloc_max_bytes.restype = SZ
    lib.moe_expert_ffn_noalloc_max_bytes.argtypes = []
    lib.fp8_block_gemm.restype = I32
    lib.fp8_block_gemm.argtypes = [P, P, P, P, I32, I32, I32, P, I32, P]
    lib.moe_shared_expert_workspace_bytes.restype = SZ
    lib.moe_shared_expert_workspace_bytes.argtypes = [I32, I32, I32]
    lib.moe_shared_expert.restype = I32
    lib.moe_shared_expert.argtypes = [P, P, I32, I32, P, P, P, P, I32, P, P, SZ, P]
    lib.moe_layer_decode1.restype = I32
    lib.moe_layer_decode1.argtypes = [P, I32, I32, P, F32, P, P, I32, P, P, P, P, I32, P, P, P, P, P, P, P, SZ, P]
    lib.moe_layer_decode1_shared_workspace_bytes.restype = SZ
    lib.moe_layer_decode1_shared_workspace_bytes.argtypes = [I32, I32, I32, I32, I32]
    lib.moe_layer_decode1_shared.restype = I32
    lib.moe_layer_decode1_shared.argtypes = [P, I32, I32, P, F32, P, P, I32, P, P, P, P, I32, P, P, P, P, I32,
                                             P, P, P, P, P, P, P, P, SZ, P]
    lib.mx_dequantize.restype = I32
    lib.mx_dequantize.argtypes = [P, P, I32, I64, I64, P, I32, P]
    lib.mx_swiglu_quantize.restype = I32
    lib.mx_swiglu_quantize.argtypes = [P, I32, I64, I64, I32, I32, P, P, P]
    lib.mx_add_rmsnorm.restype = I32
    lib.mx_add_rmsnorm.argtypes = [P, P, I32, I64, P, P, I32, I64, P, I32, I32, I32, F32, P, P, P, I32, P]
    lib.fp4_block_gemm.restype = I32
    lib.fp4_block_gemm.argtypes = [P, P, I32, P, P, I32, I32, I32, P, I32, P]
    lib.fp4_dense_ffn_workspace_bytes.restype = SZ
    lib.fp4_dense_ffn_workspace_bytes.argtypes = [I32, I32, I32, I32]
    lib.fp4_dense_ffn.restype = I32
    lib.fp4_dense_ffn.argtypes = [P, P, I32, I32, I32, P, P, P, P, I32, I32, P, I32, P, SZ, P]
    lib.moe_permute.restype = I32
    lib.moe_permute.argtypes = [P, I64, I64, P, I64, P, I32, I32, P, P, I64, P]
    lib.moe_unpermute.restype = I32
    lib.moe_unpermute.argtypes = [P, I32, I64, P, P, I32, I32, I32, P, I32, P]
    lib.moe_unpermute_grad.restype = I32
    lib.moe_unpermute_grad.argtypes = [P, I32, P, I32, I64, P, P, I32, I32, I32, P, P, P]
    lib.fp8_quantize128.restype = I32
    lib.fp8_quantize128.argtypes = [P, I32, I64, I64, I64, I64, I32, P, P, P]
    lib.fp8_swiglu_quantize128.restype = I32
    lib.fp8_swiglu_quantize128.argtypes = [P, I32, I64, I64, I32, P, P, P]
    lib.fp8_quantize128_t_cols.restype = I64
    lib.fp8_quantize128_t_cols.argtypes = [I64, I32]
    lib.fp8_quantize128_t.restype = I32
    lib.fp8_quantize128_t.argtypes = [P, I32, I64, I64, I32, P, I32, P, P, I64, P]
    lib.fp8_block128_gemm.restype = I32
    lib.fp8_block128_gemm.argtypes = [P, P, P, P, I32, I32, I32, I32, P, I32, P]
    lib.fp8_block128_grouped_gemm.restype = I32
    lib.fp8_block128_grouped_gemm.argtypes = [P, P, I32, P, P, P, I32, I32, I32, P, I32, P]
    lib.fp8_block128_grouped_wgrad.restype = I32
    lib.fp8_block128_grouped_wgrad.argtypes = [P, P, P, P, I64, P, I32, I32, I32, P, I32, P]
    lib.mx_prefetch.restype = I32
    lib.mx_prefetch.argtypes = [P, ctypes.c_uint64, ctypes.c_uint64, P]
    lib.mx_status_string.restype = ctypes.c_char_p
    lib.mx_status_string.argtypes = [I32]
    lib.mx_last_variant.restype = ctypes.c_char_p
    lib.mx_last_variant.argtypes = []
    lib.mx_set_ffn_path.restype = I32
    lib.mx_set_ffn_path.argtypes = [I32]
    lib.mx_set_layer1_single_launch.restype = I32
    lib.mx_set_layer1_single_launch.argtypes = [I32]
    lib.mx_check_requant.restype = I32
    lib.mx_check_requant.argtypes = [ctypes.c_uint32, ctypes.c_uint32, P, P]
    lib.mx_set_phase_events.restype = I32
    lib.mx_set_phase_events.argtypes = [ctypes.POINTER(ctypes.c_void_p), I32]
    _lib = lib
    return lib


def status_string(status):
    return load().mx_status_string(status).decode()


def last_variant():
    return load().mx_last_variant().decode()


def set_layer1_single_launch(on):
    """1 = moe_layer_decode1(_shared) and moe_shared_expert (T = 1) in one launch where it applies, 0 = two;
    returns the previous setting."""
    r = load().mx_set_layer1_single_launch(int(on))
    if r < 0:
        raise MXError(r, "mx_set_layer1_single_launch")
    return r


def set_ffn_path(path):
    """0 = automatic, 1 = decode kernels, 2 = prefill kernels; returns the previous setting."""
    r = load().mx_set_ffn_path(int(path))
    if r < 0:
        raise MXError(r, "mx_set_ffn_path")
    return r


# Plain ints for the c_void_p arguments: ctypes converts them by the
# argtypes, which costs less per call than building a c_void_p per argument
# (at decode sizes the Python side of a call is as long as the kernel).
def _ptr(t):
    return None if t is None else t.data_ptr()


_raw_stream = None


def _stream(stream):
    """The given stream handle, else the current torch stream of the current device (its raw handle)."""
    global _raw_stream
    if stream is not None:
        return stream
    import torch
    if _raw_stream is None:
        f = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _raw_stream = (lambda: f(torch.cuda.current_device())) if f is not None else \
            (lambda: torch.cuda.current_stream().cuda_stream)
    return _raw_stream()


def _check(status, name):
    if status != MX_OK:
        raise MXError(status, name)


# ------------------------------------------------------------------ calls
def mx_quantize(src, q, sc, fmt, stream=None):
    """Quantize src [rows, cols] (fp32 or bf16 tensor) into q / sc (uint8 tensors)."""
    import torch
    dt = {torch.float32: MX_IN_F32, torch.bfloat16: MX_IN_BF16}[src.dtype]
    cols = src.shape[-1]
    rows = src.numel() // cols if cols else 0
    _check(load().mx_quantize(_ptr(src), dt, rows, cols, fmt, _ptr(q), _ptr(sc), _stream(stream)), "mx_quantize")


def moe_router_logits_workspace_bytes(T, H, E):
    return load().moe_router_logits_workspace_bytes(T, H, E)


def moe_router_logits(hidden, w_gate, logits, ws=None, stream=None):
    """logits [T, E] fp32 = hidden [T, H] bf16 . w_gate [E, H] bf16 (ws: uint8 device tensor of
    moe_router_logits_workspace_bytes(T, H, E) bytes, or None when that size is 0)."""
    T, H = hidden.shape
    E = w_gate.shape[0]
    if w_gate.shape[1] != H or tuple(logits.shape) != (T, E):
        raise ValueError("moe_router_logits: shape mismatch")
    for t in (hidden, w_gate):
        if t.element_size() != 2 or not t.is_contiguous():
            raise ValueError("moe_router_logits: hidden and w_gate must be contiguous 16-bit (bf16) tensors")
    ws_bytes = 0 if ws is None else ws.nbytes
    _check(load().moe_router_logits(_ptr(hidden), T, H, _ptr(w_gate), E, _ptr(logits), _ptr(ws), ws_bytes,
                                    _stream(stream)), "moe_router_logits")


def moe_route_workspace_bytes(T, E, k):
    return load().moe_route_workspace_bytes(T, E, k)


def moe_route(logits, k, survival, skip_below, topk_ids, topk_w, expert_offsets, perm, slot_pos, ws, stream=None):
    T, E = logits.shape
    _check(load().moe_route(_ptr(logits), T, E, k, _ptr(survival), float(skip_below), _ptr(topk_ids), _ptr(topk_w),
                            _ptr(expert_offsets), _ptr(perm), _ptr(slot_pos), _ptr(ws), ws.nbytes,
                            _stream(stream)), "moe_route")


def moe_route_live(logits, k, survival, reuse_below, anchor, topk_ids, topk_w, expert_offsets, perm, slot_pos, ws,
                   stream=None):
    T, E = logits.shape
    _check(load().moe_route_live(_ptr(logits), T, E, k, _ptr(survival), float(reuse_below), _ptr(anchor),
                                 _ptr(topk_ids), _ptr(topk_w), _ptr(expert_offsets), _ptr(perm), _ptr(slot_pos),
                                 _ptr(ws), ws.nbytes, _stream(stream)), "moe_route_live")


def moe_expert_ffn_workspace_bytes(T, H, E, I, k):
    return load().moe_expert_ffn_workspace_bytes(T, H, E, I, k)


def moe_ws_layout(T, H, I, k):
    """Byte offsets (q, q_sc, o) of the FFN workspace regions."""
    offs = [ctypes.c_size_t() for _ in range(3)]
    _check(load().moe_ws_layout(T, H, I, k, *[ctypes.byref(o) for o in offs]), "moe_ws_layout")
    return tuple(o.value for o in offs)


def moe_expert_ffn(x, x_sc, topk_w, expert_offsets, perm, slot_pos, k, w13, w13_sc, w2, w2_sc, E, I, y, ws,
                   stream=None):
    T, H = x.shape
    _check(load().moe_expert_ffn(_ptr(x), _ptr(x_sc), T, H, _ptr(topk_w), _ptr(expert_offsets), _ptr(perm),
                                 _ptr(slot_pos), k, _ptr(w13), _ptr(w13_sc), _ptr(w2), _ptr(w2_sc), E, I, _ptr(y),
                                 _ptr(ws), ws.nbytes, _stream(stream)), "moe_expert_ffn")


def moe_expert_ffn_noalloc(x, x_sc, topk_w, expert_offsets, perm, slot_pos, k, w13, w13_sc, w2, w2_sc, E, I, y,
                           stream=None):
    """moe_expert_ffn without a caller workspace (the library's own device scratch array)."""
    T, H = x.shape
    _check(load().moe_expert_ffn_noalloc(_ptr(x), _ptr(x_sc), T, H, _ptr(topk_w), _ptr(expert_offsets), _ptr(perm),
                                         _ptr(slot_pos), k, _ptr(w13), _ptr(w13_sc), _ptr(w2), _ptr(w2_sc), E, I,
                                         _ptr(y), _stream(stream)), "moe_expert_ffn_noalloc")


def moe_expert_ffn_noalloc_max_bytes():
    return load().moe_expert_ffn_noalloc_max_bytes()


def moe_layer_decode1(logits, k, survival, skip_below, x, x_sc, w13, w13_sc, w2, w2_sc, E, I, topk_ids, topk_w,
                      expert_offsets, perm, slot_pos, y, ws, stream=None):
    """Route + routed-expert FFN of one row (logits [1, E] or [E]) in one launch (or two)."""
    H = x.shape[-1]
    _check(load().moe_layer_decode1(_ptr(logits), E, k, _ptr(survival), float(skip_below), _ptr(x), _ptr(x_sc), H,
                                    _ptr(w13), _ptr(w13_sc), _ptr(w2), _ptr(w2_sc), I, _ptr(topk_ids), _ptr(topk_w),
                                    _ptr(expert_offsets), _ptr(perm), _ptr(slot_pos), _ptr(y), _ptr(ws),
                                    ws.nbytes, _stream(stream)), "moe_layer_decode1")


def moe_layer_decode1_shared_workspace_bytes(H, E, I, k, Is):
    return load().moe_layer_decode1_shared_workspace_bytes(H, E, I, k, Is)


def moe_layer_decode1_shared(logits, k, survival, skip_below, x, x_sc, w13, w13_sc, w2, w2_sc, E, I,
                             sw13, sw13_sc, sw2, sw2_sc, topk_ids, topk_w, expert_offsets, perm, slot_pos, y,
                             y_shared, ws, stream=None):
    """moe_layer_decode1 plus the row's shared expert (sw13 FP8 [2Is, H], sw2 FP8 [H, Is] + scales) in the
    same launches (one where moe_layer_decode1 takes one and Is <= 640); y_shared [H] fp32 as moe_shared_expert."""
    H = x.shape[-1]
    Is = sw2.shape[-1]
    _check(load().moe_layer_decode1_shared(_ptr(logits), E, k, _ptr(survival), float(skip_below), _ptr(x), _ptr(x_sc),
                                           H, _ptr(w13), _ptr(w13_sc), _ptr(w2), _ptr(w2_sc), I, _ptr(sw13),
                                           _ptr(sw13_sc), _ptr(sw2), _ptr(sw2_sc), Is, _ptr(topk_ids), _ptr(topk_w),
                                           _ptr(expert_offsets), _ptr(perm), _ptr(slot_pos), _ptr(y), _ptr(y_shared),
                                           _ptr(ws), ws.nbytes, _stream(stream)),
           "moe_layer_decode1_shared")


def fp8_block_gemm(a, a_sc, w, w_sc, y, y_dtype, stream=None):
    M, K = a.shape
    N = w.shape[0]
    _check(load().fp8_block_gemm(_ptr(a), _ptr(a_sc), _ptr(w), _ptr(w_sc), M, N, K, _ptr(y), y_dtype,
                                 _stream(stream)), "fp8_block_gemm")


def moe_shared_expert_workspace_bytes(T, H, I):
    return load().moe_shared_expert_workspace_bytes(T, H, I)


def moe_shared_expert(x, x_sc, w13, w13_sc, w2, w2_sc, y, ws, stream=None):
    """y [T, H] fp32 = shared expert of x (FP8 [T, H] + scales); w13 [2I, H], w2 [H, I] FP8 + scales.
    One row (T = 1, H % 128 == 0, I <= 1024, not under graph capture) runs in one launch."""
    T, H = x.shape
    I = w2.shape[1]
    if tuple(w13.shape) != (2 * I, H) or tuple(y.shape) != (T, H):
        raise ValueError("moe_shared_expert: shape mismatch")
    _check(load().moe_shared_expert(_ptr(x), _ptr(x_sc), T, H, _ptr(w13), _ptr(w13_sc), _ptr(w2), _ptr(w2_sc), I,
                                    _ptr(y), _ptr(ws), ws.nbytes, _stream(stream)),
           "moe_shared_expert")


# ------------------------------------------- dense block in microscaled formats
# These calls check their tensors here (type, shape, layout, device): a wrong
# one raises ValueError before anything is launched.  At decode sizes the
# Python side of a call is longer than its kernel, so each call first asks one
# question that holds for right tensors; only where it does not do the checks
# below find out what is wrong, or read the strides of rows that lie apart.
class _Torch:
    """torch's names that the calls use (torch is imported with the first of them)."""

    def __init__(self):
        import torch
        self.u8, self.f32, self.bf16, self.i32 = torch.uint8, torch.float32, torch.bfloat16, torch.int32
        self.ins = {torch.float32: MX_IN_F32, torch.bfloat16: MX_IN_BF16}
        self.outs = {torch.bfloat16: MX_OUT_BF16, torch.float32: MX_OUT_F32}
        self.current_device = torch.cuda.current_device
        self.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda d: torch.cuda.current_stream(d).cuda_stream)


_torch = None


def _tn():
    global _torch
    if _torch is None:
        _torch = _Torch()
    return _torch


def _rows(name, what, t, dtypes, rows, cols):
    """The row stride of t, a 2-D tensor [rows, cols] of one of dtypes with contiguous rows."""
    if t.dim() != 2 or t.dtype not in dtypes or t.shape[0] != rows or t.shape[1] != cols:
        raise ValueError(f"{name}: {what} is {tuple(t.shape)} {t.dtype}, expected ({rows}, {cols}) {tuple(dtypes)}")
    if cols > 1 and t.stride(1) != 1 or rows > 1 and t.stride(0) < cols:
        raise ValueError(f"{name}: {what} must have contiguous rows")
    return t.stride(0) if rows > 1 else (cols + 7) // 8 * 8


def _packed(name, what, t, dtypes, shape):
    """t is contiguous, of one of dtypes and of this shape."""
    if t.dtype not in dtypes or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: {what} is {tuple(t.shape)} {t.dtype}, expected contiguous {tuple(shape)} {tuple(dtypes)}")


def _here(name, *tensors):
    """Every tensor is on the current device."""
    d = _tn().current_device()
    for t in tensors:
        if t is not None and t.get_device() != d:
            raise ValueError(f"{name}: a tensor is on {t.device}, the current device is cuda:{d}")


def _two(name, what, t):
    if t.dim() != 2:
        raise ValueError(f"{name}: {what} must be 2-D")
    return t.shape


_INT_MAX = 2**31 - 1


def _int(name, *sizes):
    """Sizes the C-ABI takes as int (ctypes would cut larger ones)."""
    if max(sizes) > _INT_MAX:
        raise ValueError(f"{name}: a size of {max(sizes)}, at most {_INT_MAX} is supported")


def _code_cols(name, fmt, cols):
    """Code bytes of a row of cols elements."""
    if fmt == MX_FMT_E4M3:
        return cols
    if fmt == MX_FMT_E2M1:
        return cols // 2
    raise ValueError(f"{name}: unknown format {fmt}")


def mx_dequantize(q, sc, fmt, out, stream=None):
    """out [rows, cols] (fp32 or bf16) = the values of codes q and scales sc."""
    name, t = "mx_dequantize", _tn()
    rows, cols = _two(name, "out", out)
    qc, d = _code_cols(name, fmt, cols), out.get_device()
    if not (q.dtype is t.u8 and sc.dtype is t.u8 and out.dtype in t.outs and q.shape == (rows, qc) and
            sc.shape == (rows, cols // 32) and q.is_contiguous() and sc.is_contiguous() and out.is_contiguous() and
            q.get_device() == d and sc.get_device() == d and t.current_device() == d):
        _packed(name, "out", out, t.outs, (rows, cols))
        _packed(name, "q", q, (t.u8,), (rows, qc))
        _packed(name, "sc", sc, (t.u8,), (rows, cols // 32))
        _here(name, q, sc, out)
    _check(load().mx_dequantize(q.data_ptr(), sc.data_ptr(), fmt, rows, cols, out.data_ptr(), t.outs[out.dtype],
                                t.raw_stream(d) if stream is None else stream), name)


def mx_swiglu_quantize(gu, q, sc, fmt, stream=None):
    """q, sc = codes of silu(gate) * up; gu [T, 2I] (fp32 or bf16, any row stride that keeps rows 16-byte
    aligned), gate in the first I columns."""
    name, t = "mx_swiglu_quantize", _tn()
    T, two_i = _two(name, "gu", gu)
    I = two_i // 2
    _int(name, I)
    qc, d, ld = _code_cols(name, fmt, I), gu.get_device(), two_i
    if not (gu.dtype in t.ins and gu.is_contiguous() and two_i == 2 * I and q.dtype is t.u8 and sc.dtype is t.u8 and
            q.shape == (T, qc) and sc.shape == (T, I // 32) and q.is_contiguous() and sc.is_contiguous() and
            q.get_device() == d and sc.get_device() == d and t.current_device() == d):
        ld = _rows(name, "gu", gu, t.ins, T, 2 * I)
        _packed(name, "q", q, (t.u8,), (T, qc))
        _packed(name, "sc", sc, (t.u8,), (T, I // 32))
        _here(name, gu, q, sc)
    _check(load().mx_swiglu_quantize(gu.data_ptr(), t.ins[gu.dtype], ld, T, I, fmt, q.data_ptr(), sc.data_ptr(),
                                     t.raw_stream(d) if stream is None else stream), name)


def mx_add_rmsnorm(x, weight, eps, residual=None, x2=None, h=None, n=None, q=None, sc=None, fmt=MX_FMT_E4M3,
                   stream=None):
    """v = (residual + x) + x2; h = v in the residual's type; n = h / sqrt(mean(h^2) + eps) * weight.
    x, x2, residual, h [T, H] fp32 or bf16 (x and x2 of one type and row stride, residual and h too; h may be
    residual); weight [H] fp32 or bf16 or None; n [T, H] bf16; q, sc the codes of n in fmt.  The outputs that are
    given are written."""
    name, t = "mx_add_rmsnorm", _tn()
    shape = _two(name, "x", x)
    T, H = shape
    _int(name, T, H)
    d, ins = x.get_device(), t.ins
    r = residual if residual is not None else h
    x_ld = r_ld = H
    if not (x.dtype in ins and x.is_contiguous() and
            (x2 is None or x2.dtype is x.dtype and x2.shape == shape and x2.is_contiguous() and x2.get_device() == d) and
            (r is None or r.dtype in ins and r.shape == shape and r.is_contiguous() and r.get_device() == d) and
            (h is None or h is r or h.dtype is r.dtype and h.shape == shape and h.is_contiguous() and
             h.get_device() == d) and
            (weight is None or weight.dtype in ins and weight.shape == (H,) and weight.is_contiguous() and
             weight.get_device() == d) and
            (n is None or n.dtype is t.bf16 and n.shape == shape and n.is_contiguous() and n.get_device() == d) and
            (q is None and sc is None or q is not None and sc is not None and q.dtype is t.u8 and sc.dtype is t.u8 and
             q.shape == (T, _code_cols(name, fmt, H)) and sc.shape == (T, H // 32) and q.is_contiguous() and
             sc.is_contiguous() and q.get_device() == d and sc.get_device() == d) and t.current_device() == d):
        x_ld = _rows(name, "x", x, ins, T, H)
        if x2 is not None and _rows(name, "x2", x2, (x.dtype,), T, H) != x_ld:
            raise ValueError(f"{name}: x2 must have x's row stride")
        if r is not None:
            r_ld = _rows(name, "residual", r, ins, T, H)
            if h is not None and h is not r and _rows(name, "h", h, (r.dtype,), T, H) != r_ld:
                raise ValueError(f"{name}: h must have the residual's row stride")
        if weight is not None:
            _packed(name, "weight", weight, ins, (H,))
        if n is not None:
            _packed(name, "n", n, (t.bf16,), (T, H))
        if (q is None) != (sc is None):
            raise ValueError(f"{name}: q and sc come together")
        if q is not None:
            _packed(name, "q", q, (t.u8,), (T, _code_cols(name, fmt, H)))
            _packed(name, "sc", sc, (t.u8,), (T, H // 32))
        _here(name, x, weight, residual, x2, h, n, q, sc)
    _check(load().mx_add_rmsnorm(x.data_ptr(), None if x2 is None else x2.data_ptr(), ins[x.dtype], x_ld,
                                 None if residual is None else residual.data_ptr(), None if h is None else h.data_ptr(),
                                 MX_IN_F32 if r is None else ins[r.dtype], r_ld,
                                 None if weight is None else weight.data_ptr(),
                                 MX_IN_F32 if weight is None else ins[weight.dtype], T, H, eps,
                                 None if n is None else n.data_ptr(), None if q is None else q.data_ptr(),
                                 None if sc is None else sc.data_ptr(), fmt,
                                 t.raw_stream(d) if stream is None else stream), name)


def fp4_block_gemm(a, a_sc, a_fmt, w, w_sc, y, stream=None):
    """y [M, N] (bf16 or fp32) = a . w^T; a codes of K elements a row in a_fmt, w E2M1 [N, K/2], scales [., K/32]."""
    name, t = "fp4_block_gemm", _tn()
    N, K = _two(name, "w", w)
    M, yn = _two(name, "y", y)
    K *= 2
    _int(name, M, N, K)
    ac, nb, d, u8 = _code_cols(name, a_fmt, K), K // 32, y.get_device(), t.u8
    if not (yn == N and y.dtype in t.outs and w.dtype is u8 and a.dtype is u8 and a_sc.dtype is u8 and w_sc.dtype is u8 and
            a.shape == (M, ac) and a_sc.shape == (M, nb) and w_sc.shape == (N, nb) and w.is_contiguous() and
            a.is_contiguous() and a_sc.is_contiguous() and w_sc.is_contiguous() and y.is_contiguous() and
            a.get_device() == d and a_sc.get_device() == d and w.get_device() == d and w_sc.get_device() == d and
            t.current_device() == d):
        _packed(name, "w", w, (u8,), (N, K // 2))
        _packed(name, "w_sc", w_sc, (u8,), (N, nb))
        _packed(name, "a", a, (u8,), (M, ac))
        _packed(name, "a_sc", a_sc, (u8,), (M, nb))
        _packed(name, "y", y, t.outs, (M, N))
        _here(name, a, a_sc, w, w_sc, y)
    _check(load().fp4_block_gemm(a.data_ptr(), a_sc.data_ptr(), a_fmt, w.data_ptr(), w_sc.data_ptr(), M, N, K,
                                 y.data_ptr(), t.outs[y.dtype], t.raw_stream(d) if stream is None else stream), name)


def fp4_dense_ffn_workspace_bytes(T, H, I, mid_fmt):
    return load().fp4_dense_ffn_workspace_bytes(T, H, I, mid_fmt)


def fp4_dense_ffn(x, x_sc, x_fmt, w13, w13_sc, w2, w2_sc, mid_fmt, y, ws, stream=None):
    """y [T, H] (bf16 or fp32) = SwiGLU FFN of x (codes in x_fmt) with E2M1 weights w13 [2I, H/2] (gate, then up),
    w2 [H, I/2]; the intermediate in mid_fmt; ws a tensor of fp4_dense_ffn_workspace_bytes(T, H, I, mid_fmt) bytes."""
    name, t = "fp4_dense_ffn", _tn()
    H, I = _two(name, "w2", w2)
    T = _two(name, "y", y)[0]
    I *= 2
    _int(name, T, H, I)
    xc, hb, ib, d, u8 = _code_cols(name, x_fmt, H), H // 32, I // 32, y.get_device(), t.u8
    if not (y.dtype in t.outs and y.shape == (T, H) and x.dtype is u8 and x_sc.dtype is u8 and w13.dtype is u8 and
            w13_sc.dtype is u8 and w2.dtype is u8 and w2_sc.dtype is u8 and x.shape == (T, xc) and
            x_sc.shape == (T, hb) and w13.shape == (2 * I, H // 2) and w13_sc.shape == (2 * I, hb) and
            w2_sc.shape == (H, ib) and x.is_contiguous() and x_sc.is_contiguous() and w13.is_contiguous() and
            w13_sc.is_contiguous() and w2.is_contiguous() and w2_sc.is_contiguous() and y.is_contiguous() and
            ws.is_contiguous() and x.get_device() == d and x_sc.get_device() == d and w13.get_device() == d and
            w13_sc.get_device() == d and w2.get_device() == d and w2_sc.get_device() == d and ws.get_device() == d and
            t.current_device() == d):
        _packed(name, "x", x, (u8,), (T, xc))
        _packed(name, "x_sc", x_sc, (u8,), (T, hb))
        _packed(name, "w13", w13, (u8,), (2 * I, H // 2))
        _packed(name, "w13_sc", w13_sc, (u8,), (2 * I, hb))
        _packed(name, "w2", w2, (u8,), (H, I // 2))
        _packed(name, "w2_sc", w2_sc, (u8,), (H, ib))
        _packed(name, "y", y, t.outs, (T, H))
        if not ws.is_contiguous():
            raise ValueError(f"{name}: ws must be contiguous")
        _here(name, x, x_sc, w13, w13_sc, w2, w2_sc, y, ws)
    _check(load().fp4_dense_ffn(x.data_ptr(), x_sc.data_ptr(), x_fmt, T, H, w13.data_ptr(), w13_sc.data_ptr(),
                                w2.data_ptr(), w2_sc.data_ptr(), I, mid_fmt, y.data_ptr(), t.outs[y.dtype],
                                ws.data_ptr(), ws.nbytes, t.raw_stream(d) if stream is None else stream), name)


# ------------------------------ experts' tokens, products with a scale for each block of 128
# Checked as the dense block's calls are: one question that holds for right
# tensors, and only where it does not the checks that find out what is wrong.
def _blocks(n):
    return -(-n // 128)


def moe_permute(x, slot_pos, out, x_sc=None, out_sc=None, stream=None):
    """out[slot_pos[t, j]] = x[t]; x [T, H] of any type with contiguous rows, out [R, H] of the same type, slot_pos int32
    [T, k]; rows that no slot names are left as they were.  x_sc [T, B] and out_sc [R, B]: the rows' scales, alike."""
    name, t = "moe_permute", _tn()
    T, H = _two(name, "x", x)
    R, k = _two(name, "out", out)[0], _two(name, "slot_pos", slot_pos)[1]
    d, size, dtype, B = x.get_device(), x.element_size(), x.dtype, 0
    ld = H
    if x_sc is not None and out_sc is not None:
        B = _two(name, "x_sc", x_sc)[1]
    if not (x.is_contiguous() and out.dtype is dtype and out.shape == (R, H) and out.is_contiguous() and
            out.get_device() == d and slot_pos.dtype is t.i32 and slot_pos.shape == (T, k) and slot_pos.is_contiguous() and
            slot_pos.get_device() == d and H > 0 and T <= _INT_MAX and
            (x_sc is None and out_sc is None or
             out_sc is not None and x_sc is not None and x_sc.shape == (T, B) and x_sc.is_contiguous() and
             x_sc.get_device() == d and out_sc.dtype is x_sc.dtype and out_sc.shape == (R, B) and out_sc.is_contiguous() and
             out_sc.get_device() == d) and t.current_device() == d):
        if (x_sc is None) != (out_sc is None):
            raise ValueError(f"{name}: x_sc and out_sc come together")
        if H == 0:
            raise ValueError(f"{name}: x has no columns")
        _int(name, T, k)
        ld = _rows(name, "x", x, (dtype,), T, H) if T > 1 else H
        if H > 1 and x.stride(1) != 1:
            raise ValueError(f"{name}: x must have contiguous rows")
        _packed(name, "out", out, (dtype,), (R, H))
        _packed(name, "slot_pos", slot_pos, (t.i32,), (T, k))
        if x_sc is not None:
            _packed(name, "x_sc", x_sc, (x_sc.dtype,), (T, B))
            _packed(name, "out_sc", out_sc, (x_sc.dtype,), (R, B))
        _here(name, x, slot_pos, out, x_sc, out_sc)
    _check(load().moe_permute(x.data_ptr(), ld * size, H * size, x_sc.data_ptr() if B else None,
                              B * x_sc.element_size() if B else 0, slot_pos.data_ptr(), T, k, out.data_ptr(),
                              out_sc.data_ptr() if B else None, R, t.raw_stream(d) if stream is None else stream), name)


def moe_unpermute(o, w, slot_pos, y, stream=None):
    """y[t] = sum_j w[t, j] o[slot_pos[t, j]] (w None: ones); o [R, H] and y [T, H] fp32 or bf16, w fp32 [T, k], slot_pos
    int32 [T, k]."""
    name, t = "moe_unpermute", _tn()
    R, H = _two(name, "o", o)
    T, k = _two(name, "slot_pos", slot_pos)
    d = o.get_device()
    if not (o.dtype in t.ins and o.is_contiguous() and y.dtype in t.outs and y.shape == (T, H) and y.is_contiguous() and
            y.get_device() == d and slot_pos.dtype is t.i32 and slot_pos.is_contiguous() and slot_pos.get_device() == d and
            (w is None or w.dtype is t.f32 and w.shape == (T, k) and w.is_contiguous() and w.get_device() == d) and
            (T | H) <= _INT_MAX and t.current_device() == d):
        _int(name, T, k, H)
        _packed(name, "o", o, t.ins, (R, H))
        _packed(name, "y", y, t.outs, (T, H))
        _packed(name, "slot_pos", slot_pos, (t.i32,), (T, k))
        if w is not None:
            _packed(name, "w", w, (t.f32,), (T, k))
        _here(name, o, w, slot_pos, y)
    _check(load().moe_unpermute(o.data_ptr(), t.ins[o.dtype], R, None if w is None else w.data_ptr(), slot_pos.data_ptr(), T, k,
                                H, y.data_ptr(), t.outs[y.dtype], t.raw_stream(d) if stream is None else stream), name)


def moe_unpermute_grad(dy, o, w, slot_pos, d_o=None, dw=None, stream=None):
    """The gradient of moe_unpermute: d_o[slot_pos[t, j]] = w[t, j] dy[t] (o's type; may be o itself), dw[t, j] =
    <dy[t], o[slot_pos[t, j]]> (fp32).  The outputs that are given are written; o may be None without dw."""
    name, t = "moe_unpermute_grad", _tn()
    T, H = _two(name, "dy", dy)
    k = _two(name, "slot_pos", slot_pos)[1]
    rows = o if o is not None else d_o
    if rows is None or d_o is None and dw is None or dw is not None and o is None:
        raise ValueError(f"{name}: d_o or dw is needed, and o for dw")
    R, d, f32, dtype = _two(name, "o", rows)[0], dy.get_device(), t.f32, rows.dtype
    if not (dy.dtype in t.ins and dy.is_contiguous() and dtype in t.ins and rows.shape == (R, H) and rows.is_contiguous() and
            rows.get_device() == d and
            (d_o is None or d_o.dtype is dtype and d_o.shape == (R, H) and d_o.is_contiguous() and d_o.get_device() == d) and
            slot_pos.dtype is t.i32 and slot_pos.shape == (T, k) and slot_pos.is_contiguous() and slot_pos.get_device() == d and
            (w is None or w.dtype is f32 and w.shape == (T, k) and w.is_contiguous() and w.get_device() == d) and
            (dw is None or dw.dtype is f32 and dw.shape == (T, k) and dw.is_contiguous() and dw.get_device() == d) and
            (T | H) <= _INT_MAX and t.current_device() == d):
        _int(name, T, k, H)
        _packed(name, "dy", dy, t.ins, (T, H))
        _packed(name, "o", rows, t.ins, (R, H))
        if d_o is not None:
            _packed(name, "d_o", d_o, (dtype,), (R, H))
        _packed(name, "slot_pos", slot_pos, (t.i32,), (T, k))
        for what, v in (("w", w), ("dw", dw)):
            if v is not None:
                _packed(name, what, v, (f32,), (T, k))
        _here(name, dy, o, w, slot_pos, d_o, dw)
    _check(load().moe_unpermute_grad(dy.data_ptr(), t.ins[dy.dtype], None if o is None else o.data_ptr(), t.ins[dtype], R,
                                     None if w is None else w.data_ptr(), slot_pos.data_ptr(), T, k, H,
                                     None if d_o is None else d_o.data_ptr(), None if dw is None else dw.data_ptr(),
                                     t.raw_stream(d) if stream is None else stream), name)


def fp8_quantize128(src, q, sc, block_rows=1, stream=None):
    """q, sc = E4M3 codes and fp32 scales of src, [rows, cols] or [count, rows, cols], fp32 or bf16, in blocks of 1 x 128
    (block_rows 1: sc [..., rows, nb]) or 128 x 128 (sc [..., ceil(rows / 128), nb]).  Rows of a 2-D src may lie apart."""
    name, t = "fp8_quantize128", _tn()
    shape = src.shape
    if len(shape) not in (2, 3):
        raise ValueError(f"{name}: src must be 2-D or 3-D")
    if block_rows not in (1, 128):
        raise ValueError(f"{name}: block_rows is {block_rows}, expected 1 or 128")
    rows, cols = shape[-2:]
    count, d, ld = shape[0] if len(shape) == 3 else 1, src.get_device(), cols
    sc_shape = tuple(shape[:-2]) + (rows if block_rows == 1 else _blocks(rows), _blocks(cols))
    if not (src.dtype in t.ins and src.is_contiguous() and q.dtype is t.u8 and q.shape == shape and q.is_contiguous() and
            q.get_device() == d and sc.dtype is t.f32 and sc.shape == sc_shape and sc.is_contiguous() and
            sc.get_device() == d and t.current_device() == d):
        if len(shape) == 3:
            _packed(name, "src", src, t.ins, shape)
        else:
            ld = _rows(name, "src", src, t.ins, rows, cols)
        _packed(name, "q", q, (t.u8,), shape)
        _packed(name, "sc", sc, (t.f32,), sc_shape)
        _here(name, src, q, sc)
    _check(load().fp8_quantize128(src.data_ptr(), t.ins[src.dtype], ld, count, rows, cols, block_rows, q.data_ptr(),
                                  sc.data_ptr(), t.raw_stream(d) if stream is None else stream), name)


def fp8_swiglu_quantize128(gu, q, sc, stream=None):
    """q [T, I], sc [T, ceil(I / 128)] = codes and fp32 scales of silu(gate) * up; gu [T, 2I] (fp32 or bf16, any row stride
    that keeps rows 16-byte aligned), gate in the first I columns."""
    name, t = "fp8_swiglu_quantize128", _tn()
    T, two_i = _two(name, "gu", gu)
    I = two_i // 2
    d, ld = gu.get_device(), two_i
    if not (gu.dtype in t.ins and gu.is_contiguous() and two_i == 2 * I and q.dtype is t.u8 and q.shape == (T, I) and
            q.is_contiguous() and q.get_device() == d and sc.dtype is t.f32 and sc.shape == (T, _blocks(I)) and
            sc.is_contiguous() and sc.get_device() == d and I <= _INT_MAX and t.current_device() == d):
        _int(name, I)
        ld = _rows(name, "gu", gu, t.ins, T, 2 * I)
        _packed(name, "q", q, (t.u8,), (T, I))
        _packed(name, "sc", sc, (t.f32,), (T, _blocks(I)))
        _here(name, gu, q, sc)
    _check(load().fp8_swiglu_quantize128(gu.data_ptr(), t.ins[gu.dtype], ld, T, I, q.data_ptr(), sc.data_ptr(),
                                         t.raw_stream(d) if stream is None else stream), name)


def fp8_quantize128_t_cols(rows, E=1):
    """Columns of codes that hold any split of rows into E groups."""
    return load().fp8_quantize128_t_cols(rows, E)


def fp8_quantize128_t(src, q, sc, offsets=None, stream=None):
    """q [cols, ld], sc [cols, ld / 128] = codes and scales of src [rows, cols] (fp32 or bf16) along its columns, transposed,
    in blocks of 128 rows; offsets (int32 [E + 1]) cuts the rows into groups that start at multiples of 128.  ld at least
    fp8_quantize128_t_cols(rows, E)."""
    name, t = "fp8_quantize128_t", _tn()
    rows, cols = _two(name, "src", src)
    q_ld = _two(name, "q", q)[1]
    E, d, ld = 1 if offsets is None else offsets.numel() - 1, src.get_device(), cols
    if not (src.dtype in t.ins and src.is_contiguous() and q_ld % 128 == 0 and q.dtype is t.u8 and q.shape == (cols, q_ld) and
            q.is_contiguous() and q.get_device() == d and sc.dtype is t.f32 and sc.shape == (cols, q_ld // 128) and
            sc.is_contiguous() and sc.get_device() == d and
            (offsets is None or offsets.dtype is t.i32 and offsets.shape == (E + 1,) and offsets.is_contiguous() and
             offsets.get_device() == d) and (rows | cols) <= _INT_MAX and t.current_device() == d):
        _int(name, rows, cols)
        if rows > 1:
            ld = _rows(name, "src", src, t.ins, rows, cols)
        else:
            _packed(name, "src", src, t.ins, (rows, cols))
        if q_ld % 128:
            raise ValueError(f"{name}: q has {q_ld} columns, a multiple of 128 is expected")
        _packed(name, "q", q, (t.u8,), (cols, q_ld))
        _packed(name, "sc", sc, (t.f32,), (cols, q_ld // 128))
        if offsets is not None:
            _packed(name, "offsets", offsets, (t.i32,), (E + 1,))
        _here(name, src, q, sc, offsets)
    _check(load().fp8_quantize128_t(src.data_ptr(), t.ins[src.dtype], ld, rows, cols,
                                    None if offsets is None else offsets.data_ptr(), E, q.data_ptr(), sc.data_ptr(), q_ld,
                                    t.raw_stream(d) if stream is None else stream), name)


def fp8_block128_gemm(a, a_sc, w, w_sc, y, stream=None):
    """y [M, N] (bf16 or fp32) = a . w^T; E4M3 codes a [M, K], w [N, K], fp32 scales a_sc [M, nb] and w_sc [ceil(N / 128),
    nb] (tiles) or [N, nb] (rows), nb = ceil(K / 128)."""
    name, t = "fp8_block128_gemm", _tn()
    N, K = _two(name, "w", w)
    M, sn = _two(name, "y", y)[0], _two(name, "w_sc", w_sc)[0]
    nb, d, u8, f32 = -(-K // 128), y.get_device(), t.u8, t.f32
    if not (y.dtype in t.outs and y.shape == (M, N) and y.is_contiguous() and a.dtype is u8 and a.shape == (M, K) and
            a.is_contiguous() and a.get_device() == d and w.dtype is u8 and w.is_contiguous() and w.get_device() == d and
            a_sc.dtype is f32 and a_sc.shape == (M, nb) and a_sc.is_contiguous() and a_sc.get_device() == d and
            w_sc.dtype is f32 and (sn == N or sn == -(-N // 128)) and w_sc.shape == (sn, nb) and w_sc.is_contiguous() and
            w_sc.get_device() == d and (M | N | K) <= _INT_MAX and t.current_device() == d):
        _int(name, M, N, K)
        _packed(name, "a", a, (u8,), (M, K))
        _packed(name, "w", w, (u8,), (N, K))
        _packed(name, "a_sc", a_sc, (f32,), (M, nb))
        _packed(name, "w_sc", w_sc, (f32,), (N if sn == N else _blocks(N), nb))
        _packed(name, "y", y, t.outs, (M, N))
        _here(name, a, a_sc, w, w_sc, y)
    _check(load().fp8_block128_gemm(a.data_ptr(), a_sc.data_ptr(), w.data_ptr(), w_sc.data_ptr(), 1 if sn == N else 128, M, N, K,
                                    y.data_ptr(), t.outs[y.dtype], t.raw_stream(d) if stream is None else stream), name)


def fp8_block128_grouped_gemm(a, a_sc, w, w_sc, offsets, y, stream=None):
    """y[r] = a[r] . w[e]^T for rows r in [offsets[e], offsets[e + 1]); a [R, K], a_sc [R, nb], w [E, N, K], w_sc [E,
    ceil(N / 128), nb], offsets int32 [E + 1], y [R, N] bf16 or fp32.  Rows behind offsets[E] are left as they were."""
    name, t = "fp8_block128_grouped_gemm", _tn()
    if w.dim() != 3:
        raise ValueError(f"{name}: w must be 3-D")
    E, N, K = w.shape
    R = _two(name, "y", y)[0]
    nb, d, u8, f32 = -(-K // 128), y.get_device(), t.u8, t.f32
    if not (y.dtype in t.outs and y.shape == (R, N) and y.is_contiguous() and a.dtype is u8 and a.shape == (R, K) and
            a.is_contiguous() and a.get_device() == d and w.dtype is u8 and w.is_contiguous() and w.get_device() == d and
            a_sc.dtype is f32 and a_sc.shape == (R, nb) and a_sc.is_contiguous() and a_sc.get_device() == d and
            w_sc.dtype is f32 and w_sc.shape == (E, -(-N // 128), nb) and w_sc.is_contiguous() and w_sc.get_device() == d and
            offsets.dtype is t.i32 and offsets.shape == (E + 1,) and offsets.is_contiguous() and offsets.get_device() == d and
            (R | N | K) <= _INT_MAX and t.current_device() == d):
        _int(name, R, N, K)
        _packed(name, "a", a, (u8,), (R, K))
        _packed(name, "w", w, (u8,), (E, N, K))
        _packed(name, "a_sc", a_sc, (f32,), (R, nb))
        _packed(name, "w_sc", w_sc, (f32,), (E, _blocks(N), nb))
        _packed(name, "offsets", offsets, (t.i32,), (E + 1,))
        _packed(name, "y", y, t.outs, (R, N))
        _here(name, a, a_sc, w, w_sc, offsets, y)
    _check(load().fp8_block128_grouped_gemm(a.data_ptr(), a_sc.data_ptr(), R, w.data_ptr(), w_sc.data_ptr(), offsets.data_ptr(), E,
                                            N, K, y.data_ptr(), t.outs[y.dtype],
                                            t.raw_stream(d) if stream is None else stream), name)


def fp8_block128_grouped_wgrad(a, a_sc, b, b_sc, offsets, dw, stream=None):
    """dw[e] = a . b^T over expert e's columns; a [N, ld] + a_sc [N, ld / 128] and b [K, ld] + b_sc as fp8_quantize128_t makes
    them with these offsets (int32 [E + 1]); dw [E, N, K] bf16 or fp32."""
    name, t = "fp8_block128_grouped_wgrad", _tn()
    if dw.dim() != 3:
        raise ValueError(f"{name}: dw must be 3-D")
    E, N, K = dw.shape
    ld = _two(name, "a", a)[1]
    nb, d, u8, f32 = ld // 128, dw.get_device(), t.u8, t.f32
    if not (dw.dtype in t.outs and ld % 128 == 0 and dw.is_contiguous() and a.dtype is u8 and a.shape == (N, ld) and
            a.is_contiguous() and a.get_device() == d and b.dtype is u8 and b.shape == (K, ld) and b.is_contiguous() and
            b.get_device() == d and a_sc.dtype is f32 and a_sc.shape == (N, nb) and a_sc.is_contiguous() and
            a_sc.get_device() == d and b_sc.dtype is f32 and b_sc.shape == (K, nb) and b_sc.is_contiguous() and
            b_sc.get_device() == d and offsets.dtype is t.i32 and offsets.shape == (E + 1,) and offsets.is_contiguous() and
            offsets.get_device() == d and (N | K | ld) <= _INT_MAX and t.current_device() == d):
        _int(name, N, K, ld)
        if ld % 128:
            raise ValueError(f"{name}: a has {ld} columns, a multiple of 128 is expected")
        _packed(name, "a", a, (u8,), (N, ld))
        _packed(name, "b", b, (u8,), (K, ld))
        _packed(name, "a_sc", a_sc, (f32,), (N, nb))
        _packed(name, "b_sc", b_sc, (f32,), (K, nb))
        _packed(name, "offsets", offsets, (t.i32,), (E + 1,))
        _packed(name, "dw", dw, t.outs, (E, N, K))
        _here(name, a, a_sc, b, b_sc, offsets, dw)
    _check(load().fp8_block128_grouped_wgrad(a.data_ptr(), a_sc.data_ptr(), b.data_ptr(), b_sc.data_ptr(), ld, offsets.data_ptr(),
                                             E, N, K, dw.data_ptr(), t.outs[dw.dtype],
                                             t.raw_stream(d) if stream is None else stream), name)


def prefetch(t, chunk_bytes=0, stream=None, nbytes=None):
    """Read tensor t's bytes (or its first nbytes) into cache; see mx_prefetch."""
    n = t.numel() * t.element_size() if nbytes is None else nbytes
    _check(load().mx_prefetch(_ptr(t), n, chunk_bytes, _stream(stream)), "mx_prefetch")


def check_requant(lo, hi, mismatches, stream=None):
    """Add to mismatches (int64 device tensor of one element) the number of
    finite floats with magnitude bits in [lo, hi), both signs, whose E4M3 code
    from the FFN's hardware conversion differs from the quantize encoder's."""
    _check(load().mx_check_requant(lo, hi, _ptr(mismatches), _stream(stream)), "mx_check_requant")


def set_ffn_diag(h):
    """Have this thread's later FFN calls also write their fp32 gate/up values
    into h (float32 device tensor of at least T*k*2I elements); None stops it."""
    if h is None:
        _check(load().mx_set_ffn_diag(None, 0), "mx_set_ffn_diag")
        return
    _check(load().mx_set_ffn_diag(_ptr(h), h.numel() * h.element_size()), "mx_set_ffn_diag")


def set_phase_events(events):
    """Record torch.cuda.Event objects (4, created with enable_timing=True) at
    the phase boundaries of this thread's later moe_expert_ffn calls: before
    the first kernel, after gate/up, after the down projection, after the last
    kernel.  None stops the recording."""
    if events is None:
        _check(load().mx_set_phase_events(None, 0), "mx_set_phase_events")
        return
    for e in events:
        e.record()                                   # materialise the HIP event handle
    arr = (ctypes.c_void_p * 4)(*[e.cuda_event for e in events])
    _check(load().mx_set_phase_events(arr, 4), "mx_set_phase_events")
