"""Microscaled 4-bit floats in plain numpy/f64, and the products of two such matrices.  Codes are
found by comparing distances on the grid, block by block; nothing is shared with the HIP path."""

from __future__ import annotations

import math

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x):
    """(q uint8 [rows, k/2], e uint8 [rows, k/32]) of x [rows, k]: scale 2^(floor(log2 max|x|) - 2), at
    least 2^-127, codes the nearest of the grid with ties to the even code; 255 and zeros for a
    block with an infinity or a NaN."""
    x = np.asarray(x, dtype=np.float64)
    rows, k = x.shape
    q, e = np.zeros((rows, k // 2), np.uint8), np.zeros((rows, k // 32), np.uint8)
    for r in range(rows):
        for b in range(k // 32):
            v = x[r, 32 * b:32 * b + 32]
            if not np.isfinite(v).all():
                e[r, b] = 255
                continue
            top = float(np.abs(v).max())
            exp = max(math.frexp(top)[1] - 3, -127) if top > 0 else -127     # top in [2^(exp+2), 2^(exp+3))
            e[r, b] = exp + 127
            a = np.ldexp(np.abs(v), -exp)
            dist = np.abs(a[:, None] - GRID)
            near = dist == dist.min(axis=1, keepdims=True)      # a tie: two codes, one of them even
            even = near & (np.arange(8) % 2 == 0)
            code = np.where(near.sum(axis=1) > 1, even.argmax(axis=1), near.argmax(axis=1)) + 8 * np.signbit(v)
            q[r, 16 * b:16 * b + 16] = code[0::2] + 16 * code[1::2]
    return q, e


def dequantize(q, e):
    """f64 values [.., k] of codes [.., k/2] and scales [.., k/32]; NaN for scale 255."""
    q, e = np.asarray(q), np.asarray(e)
    code = np.stack([q & 15, q >> 4], axis=-1).reshape(q.shape[:-1] + (2 * q.shape[-1],))
    v = np.where(code & 8, -1.0, 1.0) * GRID[code & 7]
    s = np.where(e == 255, np.nan, np.ldexp(1.0, np.where(e == 255, 0, e.astype(np.int64) - 127)))
    return v * np.repeat(s, 32, axis=-1)


def gemm(wq, we, xq, xe, s=None):
    """(dst [n, m], tol [n, m]) in f64.  Products of codes and scales are exact in f32 (4 bits by a
    power of two each); k of them are summed in some order in f32, each addition off by at most
    2^-24 of a partial sum, which is at most sum |w x|: k - 1 of them, the parts of up to 16 waves
    and the last multiplication stay below (k + 16) 2^-24 sum |w x|."""
    w, x = dequantize(wq, we), dequantize(xq, xe)
    f = np.ones(len(x)) if s is None else np.asarray(s, dtype=np.float64)
    return f[:, None] * (x @ w.T), np.abs(f)[:, None] * (w.shape[1] + 16) * 2.0 ** -24 * (np.abs(x) @ np.abs(w).T)
