"""Pins of the oracle's expert layer: a hand-worked case, ties, and special
cases that reduce to a dense layer."""
import numpy as np

import oracle


def test_hand_worked_token():
    # two experts of one hidden unit, d = 2; scores are x itself
    x = np.array([[1.0, 2.0]])
    Wr = np.eye(2)
    W_gu = np.array([[[1.0, 0.0], [0.0, 1.0]], [[0.0, 1.0], [1.0, 0.0]]])  # expert 0: g = x0, u = x1; 1: g = x1, u = x0
    W_d = np.array([[[1.0, 0.0]], [[0.0, 1.0]]])
    y, idx, gate = oracle.moe_layer(x, Wr, W_gu, W_d, 2, True)
    assert idx.tolist() == [[1, 0]]
    p = 1.0 / (1.0 + np.exp(-1.0))
    assert np.allclose(gate, [[p, 1 - p]])
    silu = lambda v: v / (1 + np.exp(-v))  # noqa: E731
    assert np.allclose(y, [[(1 - p) * silu(1.0) * 2.0, p * silu(2.0) * 1.0]])
    _, _, g1 = oracle.moe_layer(x, Wr, W_gu, W_d, 1, True)
    _, _, g0 = oracle.moe_layer(x, Wr, W_gu, W_d, 1, False)
    assert np.allclose(g1, 1.0) and np.allclose(g0, p)


def test_equal_scores_take_the_lower_index():
    x = np.ones((1, 4))
    Wr = np.zeros((6, 4))
    Wr[4] = 1.0
    _, idx, gate = oracle.moe_layer(x, Wr, np.zeros((6, 4, 2)), np.zeros((6, 1, 4)), 3, True)
    assert idx.tolist() == [[4, 0, 1]]
    assert np.isclose(gate.sum(), 1.0)


def test_equal_experts_are_one_dense_layer():
    rng = np.random.default_rng(2)
    x, gu, dn = rng.standard_normal((3, 8)), rng.standard_normal((8, 10)), rng.standard_normal((5, 8))
    y, _, _ = oracle.moe_layer(x, rng.standard_normal((4, 8)), np.stack([gu] * 4), np.stack([dn] * 4), 3, True)
    a = x @ gu
    assert np.allclose(y, (a[:, :5] / (1 + np.exp(-a[:, :5])) * a[:, 5:]) @ dn)
