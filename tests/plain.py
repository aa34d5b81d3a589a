"""Plain implementations in 64 bits of the row operators, the 4-bit format and the experts' FFN,
for the tests. They share no code with the library."""

from __future__ import annotations

import numpy as np

U = 2.0 ** -24                       # half a step of fp32, relative
LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def hadamard() -> np.ndarray:
    i = np.arange(128)
    return 1.0 - 2.0 * (np.array([bin(v).count("1") & 1 for v in range(128)])[i[:, None] & i[None, :]])


def wht32(x: np.ndarray) -> np.ndarray:
    """H x per 128-block in fp32, spans 1, 2, ..., 64, each (a, b) -> (a + b, a - b)."""
    v = np.ascontiguousarray(x, dtype=np.float32).reshape(-1, 128).copy()
    h = 1
    while h < 128:
        w = v.reshape(-1, 128 // (2 * h), 2, h)
        a, b = w[:, :, 0].copy(), w[:, :, 1].copy()
        w[:, :, 0], w[:, :, 1] = a + b, a - b
        h *= 2
    return v.reshape(x.shape)


def quant_i8(u: np.ndarray):
    """(codes, amax) of fp32 rows u per 128-block, in fp32 as the operator's definition states."""
    b = u.reshape(u.shape[0], -1, 128)
    amax = np.abs(b).max(-1, keepdims=True)
    amax = np.where(amax < np.float32(2.0 ** -100), np.float32(0), amax)
    inv = np.float32(127) / np.where(amax > 0, amax, np.float32(1))
    q = np.where(amax > 0, np.rint(b * inv), 0)
    return q.astype(np.int8).reshape(u.shape), amax[..., 0]


def mx_quant(x: np.ndarray):
    """(codes [m][k/2], scale bytes [m][k/32]) of fp32 rows (every fp32 value is exact in 64 bits)."""
    m, k = x.shape
    b = x.astype(np.float64).reshape(m, k // 32, 32)
    with np.errstate(invalid="ignore", divide="ignore"):
        amax = np.abs(b).max(-1)
        bad = ~np.isfinite(b).all(-1)
        zero = ~bad & (amax < 2.0 ** -124)
        e = np.floor(np.log2(np.where(bad | zero, 1.0, amax)))
        a = np.where(bad[..., None] | zero[..., None], 0.0, np.abs(b)) / (2.0 ** (e - 2))[..., None]
    # nearest level; a tie goes to the even code
    idx = np.zeros(a.shape, dtype=np.int64)
    for i, mid in enumerate((LEVELS[1:] + LEVELS[:-1]) / 2):
        idx += (a > mid) | ((a == mid) & (i % 2 == 1))
    sign = np.where(bad[..., None] | zero[..., None], 0, np.signbit(b)).astype(np.int64)
    code = (idx | sign << 3).reshape(m, k).astype(np.uint8)
    scale = np.where(bad, 255, np.where(zero, 0, e - 2 + 127)).astype(np.uint8)
    return code[:, 0::2] | code[:, 1::2] << 4, scale


def mx_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    m, nb = scales.shape
    c = np.stack([codes & 15, codes >> 4], -1).reshape(m, nb, 32)
    v = LEVELS[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (v * s[..., None]).reshape(m, nb * 32)


def weights(w) -> np.ndarray:
    """A synth.PackedMatrix in 64 bits."""
    bits = 2 if w.fmt == 0 else 1
    c = w.codes.reshape(w.n, -1, 1) >> np.arange(0, 8, bits) & (2 ** bits - 1)
    t = np.array([0, 1, -1, 0])[c] if w.fmt == 0 else 2 * c.astype(np.int64) - 1
    return t.reshape(w.n, -1, 128) * w.scales_f32().astype(np.float64).reshape(w.n, -1, 1)
