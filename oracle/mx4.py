"""Plain numpy oracle of the microscaled 4-bit operators (float64, no shared code with the HIP path).

A block is 32 consecutive values of a row. Its scale is 2^e, e = max(floor(log2 max|x|) - 2, -127), and each value
is rounded to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 times the scale, ties to the even code, saturating at 6
times the scale. A block with an Inf or a NaN is NaN as a whole.
"""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x: np.ndarray):
    """x [rows, k] -> (code [rows, kp] 0..15, scale byte [rows, kp/32]), kp = k rounded up to 128."""
    x = np.asarray(x, dtype=np.float64)
    rows, k = x.shape
    kp = -(-k // 128) * 128
    b = np.zeros((rows, kp))
    b[:, :k] = x
    b = b.reshape(rows, kp // 32, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    top = np.abs(b).max(-1)
    e = np.where(top > 0, np.frexp(top)[1] - 3, -127)  # frexp: top = m 2^f with m in [.5, 1)
    e = np.maximum(e, -127)
    v = np.ldexp(b, -e[..., None])
    a = np.abs(v)
    dist = np.abs(np.minimum(a, 6.0)[..., None] - GRID)
    near = dist.min(-1, keepdims=True)
    # of the (at most two) nearest grid values the one with the even code
    code = np.where(dist == near, np.arange(8) % 2 * 100 + np.arange(8), 1000).argmin(-1)
    code = code + 8 * np.signbit(v)
    s = np.where(bad, 255, e + 127)
    code = np.where(bad[..., None], 0, code)
    return code.reshape(rows, kp).astype(np.uint8), s.astype(np.uint8)


def values(code: np.ndarray, s: np.ndarray, k: int) -> np.ndarray:
    """The values [rows, k] of codes and scale bytes."""
    v = np.where(code & 8, -1.0, 1.0) * GRID[code & 7]
    scale = np.where(s == 255, np.nan, np.ldexp(1.0, s.astype(np.int64) - 127))
    return (v.reshape(v.shape[0], -1, 32) * scale[..., None]).reshape(v.shape)[:, :k]


def roundtrip(x: np.ndarray) -> np.ndarray:
    return values(*quantize(x), x.shape[1])


def store(code: np.ndarray, s: np.ndarray):
    """(codes, scales) in the stored layout of include/vggt3.h."""
    rows, nb = s.shape
    tiles = np.zeros((-(-rows // 64), nb // 4, 64, 4), dtype=np.uint8)
    for row in range(rows):
        for blk in range(nb):
            tiles[row // 64, blk // 4, 16 * (blk % 4) + row % 16, row % 64 // 16] = s[row, blk]
    return code[:, 0::2] | code[:, 1::2] << 4, tiles


def load(codes: np.ndarray, tiles: np.ndarray):
    """Inverse of store."""
    rows = codes.shape[0]
    code = np.stack([codes & 15, codes >> 4], -1).reshape(rows, -1)
    nb = code.shape[1] // 32
    s = np.zeros((rows, nb), dtype=np.uint8)
    for row in range(rows):
        for blk in range(nb):
            s[row, blk] = tiles[row // 64, blk // 4, 16 * (blk % 4) + row % 16, row % 64 // 16]
    return code, s


def matmul(a: np.ndarray, w: np.ndarray) -> np.ndarray:
    """a [m, k] times w [n, k] transposed, of values that are exact already."""
    return np.asarray(a, np.float64) @ np.asarray(w, np.float64).T


def swiglu(q: np.ndarray, wg: np.ndarray, wu: np.ndarray) -> np.ndarray:
    g = matmul(q, wg)
    return g / (1.0 + np.exp(-g)) * matmul(q, wu)


def read(q: np.ndarray, wg: np.ndarray, wu: np.ndarray, wd: np.ndarray) -> np.ndarray:
    """The read with every operand in 4 bits: q is quantised, the weights are given as values."""
    return matmul(roundtrip(swiglu(roundtrip(q), wg, wu)), wd)
