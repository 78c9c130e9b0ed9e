"""Pins of the decode-step oracle (oracle/step.py): closed forms and brute force on the CPU."""

import math

import numpy as np
import pytest

from oracle import ref, step


def test_q8_rows_agree_with_the_q8_1_oracle_and_closed_forms():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(5, 96)).astype(np.float32)
    q, d = step.q8_rows(x, 32)
    rq, rd = ref.quantize_q8_1(x, 96)
    assert np.array_equal(q, rq.reshape(q.shape)) and np.array_equal(d, rd.reshape(d.shape))
    # a power-of-two scale: the codes come back, halves go away from zero
    row = np.zeros(32, dtype=np.float32)
    row[:5] = [127, 2.5, -2.5, 0.5, -0.49]
    q, d = step.q8_rows(row[None], 32)
    assert d[0, 0] == 1 and q[0, :5].tolist() == [127, 3, -3, 1, 0]
    q, d = step.q8_rows(np.zeros((1, 64), np.float32), 64)
    assert not q.any() and not d.any()
    q, d = step.q8_rows(np.full((1, 32), 1e-39, np.float32), 32)   # 1/d would overflow
    assert not q.any() and not d.any()


def test_extend_small_case_by_hand():
    # pages of 4: sequence 0 has 5 tokens in pages 9, 8 and gets 4 more (one page), 1 is new (6 tokens:
    # two pages), 2 gets one token inside its page, 3 asks for a page that is not there any more
    table = np.array([[9, 8, -1, -1], [-1] * 4, [3, -1, -1, -1], [2, -1, -1, -1]])
    t, lens, slots, pos, used = step.extend(table, [5, 0, 2, 4], [4, 6, 1, 1], [7, 6, 5], 4, 14)
    assert t.tolist() == [[9, 8, 7, -1], [6, 5, -1, -1], [3, -1, -1, -1], [2, -1, -1, -1]]
    assert lens.tolist() == [9, 6, 3, 4] and used == 4
    assert pos.tolist() == [5, 6, 7, 8, 0, 1, 2, 3, 4, 5, 2, 4, -1, -1]
    assert slots.tolist() == [33, 34, 35, 28, 24, 25, 26, 27, 20, 21, 14, -1, -1, -1]


@pytest.mark.parametrize("group", [1, 3])
def test_attention_against_per_element_sums(group):
    rng = np.random.default_rng(2)
    n_kv, d, n = 2, 8, 7
    q, k, v = (rng.normal(size=s) for s in ((n_kv * group, d), (n, n_kv, d), (n, n_kv, d)))
    out, lse, tol = step.attention(q, k, v, 0.3)
    for h in range(n_kv * group):
        w = [math.exp(0.3 * math.fsum(q[h, x] * k[t, h // group, x] for x in range(d))) for t in range(n)]
        assert math.isclose(lse[h], math.log(math.fsum(w)), rel_tol=1e-13)
        for x in range(d):
            want = math.fsum(w[t] * v[t, h // group, x] for t in range(n)) / math.fsum(w)
            assert math.isclose(out[h, x], want, rel_tol=1e-12, abs_tol=1e-14)
    assert (tol > 0).all() and (tol < 1e-4).all()
    out, lse, _ = step.attention(q, k[:0], v[:0], 0.3)
    assert not out.any() and (lse == -np.inf).all()


def test_attention_tolerance_rejects_planted_mistakes():
    """A dropped token, a head off by one and a wrong scale are far outside the bound."""
    rng = np.random.default_rng(3)
    q, k, v = rng.normal(size=(4, 64)), rng.normal(size=(40, 2, 64)), rng.normal(size=(40, 2, 64))
    out, _, tol = step.attention(q, k, v, 0.125)
    for wrong in (step.attention(q, k[:-1], v[:-1], 0.125)[0], step.attention(q, k[:, ::-1], v, 0.125)[0],
                  step.attention(q, k, v, 0.1251)[0]):
        assert (np.abs(wrong - out) > tol).mean() > 0.5


def test_rmsnorm_closed_form():
    y, inv = step.rmsnorm(np.full((1, 8), 3.0), np.arange(8.0), 0.0)
    assert np.allclose(y[0], np.arange(8.0)) and np.isclose(inv[0, 0], 1 / 3)
    y, inv = step.rmsnorm(np.zeros((1, 8)), np.ones(8), 1e-6)
    assert not y.any() and np.isclose(inv[0, 0], 1e3)
