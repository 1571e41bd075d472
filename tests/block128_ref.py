"""Plain 64-bit forms of the experts' tokens and of FP8 products with a scale for each block of 128, for the tests."""
import numpy as np
import torch

from gpu_common import E4M3_MAG

BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
B = 128


def blocks(n):
    return -(-n // B)


def decode(q):
    """E4M3 codes -> float64 values."""
    q = np.asarray(q)
    mag = np.append(E4M3_MAG, np.nan)[q & 0x7F]
    return np.where(q & 0x80, -mag, mag)


def encode(v):
    """float64 values -> E4M3 codes by search: the nearest, ties to the even code, saturating."""
    a = np.abs(v)
    mids = (E4M3_MAG[1:] + E4M3_MAG[:-1]) / 2
    low, high = np.searchsorted(mids, a, "left"), np.searchsorted(mids, a, "right")
    return (np.where(low % 2 == 0, low, high) | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def cast(v, rows, cols):
    """float64 [R, C] -> (codes [R, C], scales fp32 [ceil(R / rows), ceil(C / cols)])."""
    R, C = v.shape
    nr, nc = -(-R // rows), -(-C // cols)
    q, sc = np.zeros((R, C), np.uint8), np.zeros((nr, nc), np.float32)
    for i in range(nr):
        for j in range(nc):
            b = v[i * rows:(i + 1) * rows, j * cols:(j + 1) * cols]
            s = np.float32(max(np.abs(b).max(), 2.0 ** -60)) / np.float32(448)
            sc[i, j] = s
            q[i * rows:(i + 1) * rows, j * cols:(j + 1) * cols] = encode(b / np.float64(s))
    return q, sc


def typed(v, dtype):
    """(device tensor of dtype, its values in float64)."""
    t = torch.from_numpy(np.ascontiguousarray(v, np.float32)).to(dtype)
    return t.cuda(), t.double().numpy()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def wide(q, sc, rows):
    """Codes [R, C] and scales of blocks rows x 128 -> float64 values."""
    R, C = q.shape
    return decode(q) * np.repeat(np.repeat(np.asarray(sc, np.float64), rows, 0)[:R], B, 1)[:, :C]


def whole_codes(rng, rows, cols, most=8):
    """Codes of whole numbers -most .. most: products of them are exact in the matrix cores."""
    return encode(rng.integers(-most, most + 1, (rows, cols)).astype(np.float64))


def short_scales(rng, rows, cols):
    """fp32 scales of four bits, so that what the products are multiplied with is exact in float64."""
    return ((1 + rng.integers(0, 8, (rows, cols)) / 8) * 2.0 ** rng.integers(-2, 3, (rows, cols))).astype(np.float32)


def in_order(a, a_sc, w, w_sc, w_rows):
    """The product as its kernels are to add it: one fp32 fma per block, in order (fp32 [M, N]).  Every step is exact in
    float64 before its rounding: a block's sum of whole numbers has up to 14 bits, two scales 8, 60 bits of range in all."""
    av, wv = decode(a), decode(w)
    s_w = np.repeat(np.asarray(w_sc, np.float64), w_rows, 0)[:len(w)]
    acc = np.zeros((len(a), len(w)), np.float32)
    for b in range(blocks(a.shape[1])):
        k = slice(b * B, (b + 1) * B)
        p = av[:, k] @ wv[:, k].T
        acc = (acc.astype(np.float64) + p * (np.asarray(a_sc, np.float64)[:, b, None] * s_w[None, :, b])).astype(np.float32)
    return acc


def bf16(v):
    return torch.from_numpy(np.ascontiguousarray(v, np.float32)).to(BF16).float().numpy()


def columns(v, bounds, ld):
    """float64 [R, C], rows in groups -> (codes [C, ld], scales [C, ld / 128], first columns); zeros elsewhere."""
    q, sc = np.zeros((v.shape[1], ld), np.uint8), np.zeros((v.shape[1], ld // B), np.float32)
    at = [0]
    for a, b in zip(bounds, bounds[1:]):
        n = blocks(b - a)
        if n:
            c = at[-1]
            q[:, c * B:c * B + b - a], sc[:, c:c + n] = cast(v[a:b].T, 1, B)
        at.append(at[-1] + n)
    return q, sc, at


def plan(rng, T, k, E, live=1.0):
    """(slot_pos int32 [T, k], bounds): pairs sorted by expert, then token; rows that are not live are nowhere."""
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    alive = rng.random(T) < live
    key = np.where(alive[:, None], ids, E).ravel()
    order = np.argsort(key, kind="stable")
    pos = np.empty(T * k, np.int64)
    pos[order] = np.arange(T * k)
    slot_pos = np.where(alive[:, None], pos.reshape(T, k), -1).astype(np.int32)
    return slot_pos, np.concatenate([[0], np.cumsum(np.bincount(key, minlength=E + 1)[:E])]).astype(int)
