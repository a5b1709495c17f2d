"""Pins of the oracle's 4-bit rows, attention weights and eviction: worked
examples and closed forms."""
import math

import numpy as np
import pytest

from oracle import serving_oracle as so


def test_e2m1_by_all_neighbours():
    vals = np.array(so.E2M1)
    x = np.linspace(-7, 7, 28001)                    # steps of 1/2000: every border among them
    got = np.where(so.e2m1(x) & 8, -1, 1) * vals[so.e2m1(x) & 7]
    d = np.abs(np.abs(x)[:, None] - vals)
    assert np.allclose(np.abs(np.abs(x) - np.abs(got)), d.min(-1))
    tie = np.isclose(d, d.min(-1, keepdims=True), atol=1e-9).sum(-1) == 2
    assert tie.sum() == 14 and not (so.e2m1(x)[tie] & 1).any()
    assert np.array_equal(np.signbit(x), (so.e2m1(x) & 8) > 0)


def test_quantise4_worked_example():
    row = np.zeros(32)
    row[:4] = [6.0, -3.0, 1.0, 0.25]
    row[16] = 12.0
    c, b, s = so.quantise4(row[None])
    # 12 <= 2688 s: s = 2^-7 (21 at most); blocks 6 * 128 / 6 and 12 * 128 / 6
    assert s[0] == 2.0 ** -7 and list(b[0]) == [128.0, 256.0]
    assert list(c[0, :4]) == [7, 13, 2, 0] and c[0, 16] == 7
    assert np.array_equal(so.values4(c, b, s)[0][[0, 1, 2, 3, 16]], [6.0, -3.0, 1.0, 0.0, 12.0])


@pytest.mark.parametrize("seed", range(4))
def test_quantise4_is_near(seed):
    x = np.random.default_rng(seed).standard_normal((50, 64)) * 10.0 ** np.random.default_rng(seed).uniform(-20, 20, (50, 1))
    c, b, s = so.quantise4(x)
    y = so.values4(c, b, s)
    top = np.repeat(np.abs(x).reshape(50, 4, 16).max(-1), 16, -1)
    # half of the widest step (2 of 6) and the block scale's rounding, 2^-4
    assert np.all(np.abs(x - y) <= top * (1 / 6 + 2.0 ** -4))
    assert np.all(np.abs(x).max(-1) <= 2688 * s) and np.all(np.abs(x).max(-1) > 1344 * s)


def test_weights_add_up():
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((6, 16)), rng.standard_normal((9, 2, 16))
    w = so.attention_weights(q, k)
    assert np.allclose(w.sum(0), 3.0) and w.shape == (9, 2)
    one = so.attention_weights(np.zeros((2, 16)), k)
    assert np.allclose(one, 1 / 9)
    assert so.attention_weights(q, k[:0]).shape == (0, 2)


def test_stays_worked_examples():
    w = [5.0, 1.0, 3.0, 1.0, 2.0, 0.0]
    assert so.stays(w, 3, 0) == [0, 2, 4]
    assert so.stays(w, 4, 0) == [0, 1, 2, 4]                  # of the two ones the lower
    assert so.stays(w, 3, 2) == [0, 4, 5]
    assert so.stays(w, 2, 9) == [4, 5]
    assert so.stays(w, 0, 3) == [] and so.stays(w, 6, 0) == so.stays(w, -1, 0) == list(range(6))
    assert so.stays([0.0, -0.0, math.nan, math.inf], 2, 0) == [2, 3]
    assert so.stays([-0.0, 0.0, -1.0], 1, 0) == [0]
