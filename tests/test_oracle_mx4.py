"""Pins of the oracle's microscaled 4-bit format: hand-worked blocks, the
nearest-value property by brute force, ties, and both block directions."""
import numpy as np
import pytest

import oracle


def block(*values):
    x = np.zeros((1, 32))
    x[0, :len(values)] = values
    return x


def test_hand_worked_block():
    # max 6 -> exponent 2 - 2 = 0: scale 1
    c, s = oracle.mx4_quantize(block(6, -0.2, 0.3, 1.2, -1.4, 2.4, 2.6, 3.6, -5.2, 4.9), 1)
    assert s.tolist() == [[127]]
    assert c[0, :10].tolist() == [7, 8, 1, 2, 8 + 3, 4, 5, 6, 8 + 7, 6]
    assert oracle.mx4_values(c, s, 1)[0, :10].tolist() == [6, -0.0, 0.5, 1, -1.5, 2, 3, 4, -6, 4]


def test_ties_go_to_the_even_code():
    c, _ = oracle.mx4_quantize(block(4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -0.25), 1)
    # 0 | 1, 2, 2... : midpoints 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4
    assert c[0, :8].tolist() == [6, 0, 2, 2, 4, 4, 6, 8]
    c, _ = oracle.mx4_quantize(block(5), 1)
    assert c[0, 0] == 6  # 5 lies between 4 (code 6) and 6 (code 7)


def test_saturation_zero_and_small_blocks():
    c, s = oracle.mx4_quantize(block(7.9), 1)
    assert (c[0, 0], s[0, 0]) == (7, 127)  # 7.9 / 1 saturates at 6
    c, s = oracle.mx4_quantize(np.zeros((1, 32)), 1)
    assert s[0, 0] == 0 and not c.any()
    c, s = oracle.mx4_quantize(block(2.0 ** -140), 1)
    assert s[0, 0] == 0 and c[0, 0] == 0
    c, s = oracle.mx4_quantize(block(2.0 ** -127), 1)
    assert s[0, 0] == 0 and oracle.mx4_values(c, s, 1)[0, 0] == 2.0 ** -127
    x = block(1.0, np.inf)
    c, s = oracle.mx4_quantize(x, 1)
    assert s[0, 0] == 255 and not c.any() and np.isnan(oracle.mx4_values(c, s, 1)).all()


@pytest.mark.parametrize("axis", [0, 1])
def test_nearest_value_of_the_block_grid(axis):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((64, 96)) * np.exp2(rng.integers(-20, 20, (64, 96)))
    c, s = oracle.mx4_quantize(x, axis)
    v = oracle.mx4_values(c, s, axis)
    unit = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, axis=axis)
    grid = np.concatenate([oracle.larosa_ref.E2M1, -oracle.larosa_ref.E2M1])
    best = np.min(np.abs(x[:, :, None] - unit[:, :, None] * grid), axis=2)
    assert np.array_equal(np.abs(x - v), best)
    # the largest of a block lies in [4, 8) units
    top = np.max(np.abs(x.reshape(64, 3, 32) if axis == 1 else x.reshape(2, 32, 96)), axis=2 if axis == 1 else 1)
    ratio = top / np.ldexp(1.0, s.astype(int) - 127)
    assert np.all((ratio >= 4) & (ratio < 8))


def test_transposed_matrix_gives_transposed_blocks():
    x = np.random.default_rng(4).standard_normal((64, 32))
    c1, s1 = oracle.mx4_quantize(x, 0)
    c2, s2 = oracle.mx4_quantize(x.T, 1)
    assert np.array_equal(c1, c2.T) and np.array_equal(s1, s2.T)
