"""Plain 64-bit forms of the dense block's operators (numpy, the oracle's decode tables and casts), for the tests."""
import numpy as np
import torch

import oracle
from block_scaled_fp8xfp4_amd import mxmoe

E4M3, E2M1 = mxmoe.MX_FMT_E4M3, mxmoe.MX_FMT_E2M1
NAME = {E4M3: "e4m3", E2M1: "e2m1"}


def quantize(v, fmt):
    """fp32 [rows, cols] -> oracle's codes and scales."""
    return oracle.quantize_e4m3(v) if fmt == E4M3 else oracle.quantize_e2m1(v)


def values(q, sc, fmt):
    return oracle.dequantize(q, sc, NAME[fmt])


def bf16(v):
    """fp32 -> bf16 (nearest even) as fp32 values."""
    return torch.from_numpy(np.ascontiguousarray(v, np.float32)).to(torch.bfloat16).float().numpy()


def add_rmsnorm(x, residual, x2, weight, eps, res_bf16):
    """(h, n) as fp32 arrays; the addition in fp32, the norm in float64."""
    v = x.astype(np.float32)
    if residual is not None:
        v = residual + v
    if x2 is not None:
        v = v + x2
    h = bf16(v) if res_bf16 else v
    d = h.astype(np.float64)
    r = 1.0 / np.sqrt((d * d).mean(-1, keepdims=True) + float(np.float32(eps)))
    w = 1.0 if weight is None else weight.astype(np.float64)
    return h, (d * r * w).astype(np.float32)


def swiglu(gu):
    g, u = np.split(gu.astype(np.float64), 2, axis=-1)
    with np.errstate(over="ignore"):
        return (g / (1.0 + np.exp(-g)) * u).astype(np.float32)


def product(a, a_sc, a_fmt, w, w_sc):
    """(y, sum of |a w|) in float64."""
    av, wv = values(a, a_sc, a_fmt), values(w, w_sc, E2M1)
    return av @ wv.T, np.abs(av) @ np.abs(wv).T


def activations(rng, rows, cols, loud=True):
    v = rng.standard_normal((rows, cols))
    if loud:
        v *= np.exp(0.5 * rng.standard_normal(cols))
    return v.astype(np.float32)


def weights(rng, rows, cols):
    return quantize((rng.standard_normal((rows, cols)) * 0.02).astype(np.float32), E2M1)


def to_dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def codes_like(rows, cols, fmt, device="cuda"):
    return (torch.full((rows, cols if fmt == E4M3 else cols // 2), 0xA5, dtype=torch.uint8, device=device),
            torch.full((rows, cols // 32), 0xA5, dtype=torch.uint8, device=device))
