"""The decode-step operators in plain numpy/f64: page tables, cache rows, paged attention, RMS
norm.  Device-independent and slow; sequences one after another, tokens one page lookup each."""

from __future__ import annotations

import math

import numpy as np

SMALLEST_NORMAL = np.float32(2.0 ** -126)


def q8_rows(x, run: int):
    """(codes int8, scales float32) of the last axis in runs of `run` values: d = max|x|/127 (0 below
    the smallest normal), code = round-half-away(x * (1/d)), every step in float32 (the steps
    decide the codes)."""
    x = np.ascontiguousarray(x, dtype=np.float32)
    v = x.reshape(-1, run)
    d = (np.abs(v).max(axis=1) / np.float32(127)).astype(np.float32)
    d[d < SMALLEST_NORMAL] = 0
    inv = np.zeros_like(d)
    np.divide(np.float32(1), d, out=inv, where=d != 0)
    t = (v * inv[:, None]).astype(np.float32).astype(np.float64)
    codes = np.copysign(np.floor(np.abs(t) + 0.5), t).astype(np.int8)
    return codes.reshape(x.shape), d.reshape(x.shape[:-1] + (x.shape[-1] // run,))


def extend(table, cached, new, free, page_size: int, n_rows: int):
    """Page tables of a step: (table, seq_lens, slots, positions, pages_used), the table a copy."""
    table = np.array(table, dtype=np.int64)
    width = table.shape[1]
    seq_lens, slots, positions, used = [], [], [], 0
    for i, (c, n) in enumerate(zip(map(int, cached), map(int, new))):
        ok = c >= 0 and n >= 0 and c + n <= width * page_size
        if ok:
            have, want = math.ceil(c / page_size), math.ceil((c + n) / page_size)
            ok = want == have or used + want - have <= len(free)
            if ok:
                for r in range(want - have):
                    table[i, have + r] = free[used + r]
            used += want - have
        seq_lens.append(c + n if ok else c)
        for r in range(min(max(n, 0), n_rows - len(slots))):
            pos = c + r
            page = table[i, pos // page_size] if ok else -1
            slot = page * page_size + pos % page_size
            positions.append(pos)
            slots.append(slot if page >= 0 and slot < 2 ** 31 else -1)
    slots, positions = (v + [-1] * (n_rows - len(v)) for v in (slots, positions))
    return table, np.array(seq_lens), np.array(slots, dtype=np.int64), np.array(positions, dtype=np.int64), used


def attention(q, keys, values, scale: float):
    """One sequence: q [n_q, d], keys and values [tokens, n_kv, d] (f64).  Returns (out, lse, tol):
    tol[h, x] bounds |error| of an f32 evaluation, see below.  No tokens: zeros and -inf.

    With u = 2^-24: a score's products and sum have d + 8 roundings of at most u relative to
    A = |scale| sum|q k|, and 4u A more from q's representation in parts; its scaling and the
    difference to the maximum (in powers of two, with an offset of up to 14) add
    4u (|s - M| log2(e) + |M| log2(e) + 14) in all, the hardware exponential 4u.  That is a relative
    error e_p of each weight; the weights' parts add 4u, the two sums (tokens + 64) u each."""
    q, keys, values = (np.asarray(v, dtype=np.float64) for v in (q, keys, values))
    n_q, d = q.shape
    out, lse, tol = np.zeros((n_q, d)), np.full(n_q, -np.inf), np.zeros((n_q, d))
    if len(keys) == 0:
        return out, lse, tol
    group = n_q // keys.shape[1]
    u = 2.0 ** -24
    for h in range(n_q):
        k, v = keys[:, h // group], values[:, h // group]
        s = scale * (k * q[h]).sum(axis=1)
        a = abs(scale) * np.abs(k * q[h]).sum(axis=1)
        top = s.max()
        p = np.exp(s - top)
        out[h] = (p[:, None] * v).sum(axis=0) / p.sum()
        lse[h] = top + math.log(p.sum())
        e = (d + 12) * u * a + 4 * u * math.log2(math.e) * (np.abs(s - top) + abs(top)) + 60 * u
        ep = (p * e).sum() / p.sum()      # of the denominator
        tol[h] = ((p * (e + 4 * u))[:, None] * np.abs(v)).sum(axis=0) / p.sum()
        tol[h] += (ep + 2 * (len(k) + 64) * u) * (p[:, None] * np.abs(v)).sum(axis=0) / p.sum()
    return out, lse, tol


def lse_tol(lse, tokens: int, reach: float, d: int):
    """Bound on an f32 evaluation of the log-sum-exp: the largest score's error ((d + 12) u times
    `reach`, the largest sum |scale q k|), the sum's (tokens + 64) u, the logarithm's and the last
    roundings' 16 u (|lse| + 1)."""
    u = 2.0 ** -24
    return (d + 12) * u * reach + (tokens + 64) * u + 60 * u + 16 * u * (np.abs(lse) + 1)


def rmsnorm(h, w, eps: float):
    """y = h * w / sqrt(mean(h^2) + eps), f64, and 1/rms."""
    h, w = np.asarray(h, dtype=np.float64), np.asarray(w, dtype=np.float64)
    inv = 1.0 / np.sqrt((h * h).mean(axis=-1, keepdims=True) + eps)
    return h * inv * w, inv


def rmsnorm_rel(k: int) -> float:
    """Relative bound of an f32 evaluation with u = 2^-24.  No square goes through more than
    16 * ceil(k / 16384) + 12 roundings on its way into the sum: with 1024 threads a row, in passes
    P = ceil(k / 16384) of four times four elements a thread, its own, 3 for the others of its four,
    4P - 1 for the thread's, 6 for the wave's lanes and 15 for the 16 waves, 24 + 4P in all; with 256
    threads and up to eight times four elements 1 + 3 + 7 + 6 + 3.  The root halves them; mean, eps,
    root, inverse and the two products add at most 7."""
    terms = 16 * math.ceil(k / 16384) + 12
    return (terms / 2 + 7) * 2.0 ** -24
