"""Pins of the MXFP4 oracle: the format's own table, ties, ranges and a brute-force product."""

import math

import numpy as np
import pytest

from oracle import mxfp4


def _block(values):
    v = np.zeros(32)
    v[:len(values)] = values
    return v[None]


def test_every_code_comes_back():
    for e in (0, 1, 100, 127, 200, 252):
        codes = np.arange(16)
        q = (codes + 16 * codes[::-1]).astype(np.uint8)[None]
        x = mxfp4.dequantize(q, np.array([[e]], np.uint8))
        q2, e2 = mxfp4.quantize(x)
        assert (q2 == q).all() and e2[0, 0] == e        # the largest code, 6, fixes the scale


@pytest.mark.parametrize("value,code", [
    (0.25, 0), (0.2501, 1), (0.75, 2), (0.7499, 1), (1.25, 2), (1.26, 3), (1.75, 4), (2.5, 4), (2.51, 5), (3.5, 6),
    (3.49, 5), (5.0, 6), (5.01, 7), (6.0, 7), (7.9, 7), (-0.25, 8), (-0.75, 10), (-5.0, 14), (-7.0, 15), (-0.0, 8)])
def test_ties_go_to_the_even_code(value, code):
    q, e = mxfp4.quantize(_block([value, 4.0]) if abs(value) < 4 else _block([value, 0.0]))
    assert e[0, 0] == 127 and q[0, 0] & 15 == code


def test_scales():
    for top, byte in ((1.0, 125), (1.99, 125), (2.0, 126), (6.0, 127), (8.0, 128), (2.0 ** 127, 252), (2.0 ** -125, 0),
                      (2.0 ** -130, 0), (2.0 ** -149, 0), (0.0, 0), (math.inf, 255), (math.nan, 255)):
        q, e = mxfp4.quantize(_block([1e-30 if top > 1 else 0.0, top]))
        assert e[0, 0] == byte, top
        if byte == 255:
            assert not q.any() and np.isnan(mxfp4.dequantize(q, e)).all()
    q, e = mxfp4.quantize(_block([2.0 ** -127, 3 * 2.0 ** -128]))       # subnormal in f32
    assert mxfp4.dequantize(q, e)[0, :2].tolist() == [2.0 ** -127, 3 * 2.0 ** -128]


def test_error_is_half_a_step():
    x = np.random.default_rng(3).normal(size=(50, 96)) * 10.0 ** np.random.default_rng(4).uniform(-20, 20, (50, 1))
    q, e = mxfp4.quantize(x)
    v = mxfp4.dequantize(q, e)
    unit = np.repeat(2.0 ** (e.astype(float) - 127), 32, axis=1)
    a = np.abs(x) / unit
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    assert (a < 8).all() and (np.abs(v - x) <= np.where(a > 6, 2.0, step / 2) * unit).all()


def test_product_by_brute_force_and_a_planted_mistake():
    rng = np.random.default_rng(5)
    wq, xq = (rng.integers(0, 256, (n, 48), dtype=np.uint8) for n in (3, 2))
    we, xe = (rng.integers(120, 130, (n, 3), dtype=np.uint8) for n in (3, 2))
    got, tol = mxfp4.gemm(wq, we, xq, xe, [0.5, 3.0])

    def val(q, e, r, c):
        code = (int(q[r, c // 2]) >> (4 * (c % 2))) & 15
        man, exp = code & 1, (code >> 1) & 3
        a = man * 0.5 if exp == 0 else (1 + man / 2) * 2.0 ** (exp - 1)
        return (-a if code >> 3 else a) * 2.0 ** (int(e[r, c // 32]) - 127)

    for j in range(2):
        for i in range(3):
            want = (0.5, 3.0)[j] * math.fsum(val(wq, we, i, c) * val(xq, xe, j, c) for c in range(96))
            assert abs(got[j, i] - want) <= 1e-12 * max(1, abs(want))
    swapped = ((wq >> 4) | (wq << 4)).astype(np.uint8)
    assert (np.abs(mxfp4.gemm(swapped, we, xq, xe, [0.5, 3.0])[0] - got) > tol).any()
    assert (np.abs(mxfp4.gemm(wq, we[:, ::-1], xq, xe, [0.5, 3.0])[0] - got) > tol).any()
