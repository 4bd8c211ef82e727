"""Pins of the oracle's differential attention, key weights and eviction."""

import math

import numpy as np
import pytest

from oracle import q8


def test_difference_by_hand():
    y = q8.difference([[1.0, 2.0]], [[2.0, 2.0]], [0.5])
    assert np.array_equal(y, [[0.0, 1.0]])
    n = q8.difference([[3.0, 4.0]], [[9.0, 9.0]], [0.0], gain=[2.0, 1.0], eps=0.0)
    assert np.allclose(n, [[6.0 / math.sqrt(12.5), 4.0 / math.sqrt(12.5)]])


@pytest.mark.parametrize("alpha", [1.0, 1.5, 2.0])
def test_a_rows_weights_add_up_to_one(alpha):
    rng = np.random.default_rng(0)
    K, V, Q = rng.normal(size=(50, 8)), rng.normal(size=(50, 8)), rng.normal(size=(3, 8))
    _, tau, P, S = q8.attend(K, V, Q, alpha, first_key=[0, 7, 60])
    W = q8.key_weights(S, tau, alpha)
    assert np.allclose(W, P) and np.allclose(W.sum(1), [1.0, 1.0, 0.0])


def test_kept_keys_by_hand():
    nan, inf = float("nan"), float("inf")
    assert q8.kept_keys([5.0, 1.0, 4.0], 3) == [0, 1, 2]
    assert q8.kept_keys([0.0, 1.0, 2.0, 1.0, 1.0, 0.0], 4, sinks=1, recent=1) == [0, 1, 2, 5]
    assert q8.kept_keys([1.0, 1.0, 1.0, 1.0], 2) == [0, 1]
    assert q8.kept_keys([0.0, -0.0, -1.0, 3.0], 2) == [0, 3]
    assert q8.kept_keys([1.0, inf, nan, 2.0, -inf], 2) == [1, 2]
    assert q8.kept_keys([inf, inf, nan], 1) == [2]
    assert q8.kept_keys([9.0, 8.0, 0.0, 0.0], 2, sinks=0, recent=2) == [2, 3]


def test_evicted_pages_take_the_largest_scale():
    codes = np.arange(8.0)[:, None] * np.ones((1, 2))
    scales = [1.0, 1.0, 1.0, 1.0, 2.0, 2.0, 2.0, 2.0]
    out, now = q8.evict_rows(codes, scales, [0, 1, 3, 5, 6], 4, "int8")
    assert now == [2.0, 2.0] and out[:, 0].tolist() == [0.0, 0.0, 2.0, 5.0, 6.0]   # 0.5 and 1.5 go to even
    out, now = q8.evict_rows(codes, scales, [0, 1, 2, 3], 4, "int8")
    assert now == [1.0] and out[:, 0].tolist() == [0.0, 1.0, 2.0, 3.0]
