"""Pins of the 8-bit cache's oracle: rounding against exact rational
arithmetic, the e4m3 grid against torch's type, masks and planning by hand."""

import random
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import entmax as em
from oracle import q8


def test_e4m3_grid_is_torchs_type():
    bits = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(bits, q8.grid("e4m3"))


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_nearest_against_exact_arithmetic(code):
    rng = random.Random(1)
    g = q8.grid(code)
    for _ in range(300):
        s = float(np.float32(rng.uniform(1e-3, 1e3)))
        i = rng.randrange(len(g) - 1)
        x = float(torch.tensor((g[i] + g[i + 1]) / 2 * s * rng.choice([1.0, -1.0])).bfloat16())  # near a tie
        assert q8.nearest(x / s, code) == q8.nearest_exact(Fraction(x) / Fraction(s), code)
    ties = (g[:-1] + g[1:]) / 2
    even = np.where(np.arange(len(g) - 1) % 2 == 0, g[:-1], g[1:])
    assert np.array_equal(q8.nearest(ties, code), even)
    assert q8.nearest(1e9, code) == g[-1] and q8.nearest(-1e9, code) == -g[-1]


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_append_page_keeps_within_half_a_step(code):
    rng = np.random.default_rng(0)
    codes, scale = np.zeros((16, 8)), 0.0
    x = rng.normal(size=(16, 8)) * np.exp(rng.normal(size=(16, 1)))
    x = torch.tensor(x).bfloat16().double().numpy()
    for t in range(16):
        codes, scale, odd = q8.append_page(codes, scale, t, x[t:t + 1], code)
        assert not odd
    # a value is rounded once, and once more at each growth of the scale: steps that shrink against
    # the final one, so two half steps of the final grid bound them all (int8: a whole step of s)
    step = scale if code == "int8" else np.maximum(np.abs(codes) * scale * 2 ** -3, scale * 2 ** -9)
    growths = 16
    assert np.all(np.abs(codes * scale - x) <= step * growths / 2)
    assert scale == float(q8.scale_of(np.abs(x).max(), code))


def test_nonfinite_values_and_floor():
    c, s, odd = q8.append_page(np.zeros((4, 3)), 0.0, 0, [[np.nan, np.inf, -np.inf], [1.0, 2.0, -4.0]], "int8")
    assert odd and s == float(np.float32(4.0 / 127)) and list(c[0]) == [0.0, 127.0, -127.0]
    c, s, odd = q8.append_page(np.zeros((4, 3)), 0.0, 0, np.zeros((2, 3)), "e4m3")
    assert not odd and s == 2.0 ** -96 and not c.any()


def test_sees_by_hand():
    m = q8.sees(5, 3, window=2, prefix=1)
    assert m.astype(int).tolist() == [[1, 1, 1, 0, 0], [1, 0, 1, 1, 0], [1, 0, 0, 1, 1]]
    m = q8.sees(4, 2, first_key=[3, 3])
    assert m.astype(int).tolist() == [[0, 0, 0, 0], [0, 0, 0, 1]]
    assert q8.sees(3, 1, prefix=9).all()


def test_attend_reduces_to_softmax_and_entmax():
    rng = np.random.default_rng(2)
    K, V, Q = rng.normal(size=(9, 4)), rng.normal(size=(9, 4)), rng.normal(size=(1, 4))
    o, tau, P, _ = q8.attend(K, V, Q)
    s = (K @ Q[0]) / 2.0
    assert np.allclose(o[0], np.exp(s) @ V / np.exp(s).sum()) and np.isclose(tau[0], np.log(np.exp(s).sum()))
    o, tau, P, _ = q8.attend(K, V, Q, alpha=1.5, slope=0.3, softcap=2.0)
    z = 2.0 * np.tanh(s / 2.0) - 0.3 * np.arange(8, -1, -1)
    p, t = em.entmax(z, 1.5)
    assert np.allclose(P[0], p) and np.isclose(tau[0], t)


def test_plan_by_hand():
    table = [[-1] * 3 for _ in range(4)]
    table[2][0] = 7
    out = q8.plan([0, 0, 5, 0], table, 16, 10, [3, 4, 5], [2, 0, 9, 1, 3], [12, 17, 1, 40, 1], 80)
    t, lens, free, start, count, pos, slots, refused = out
    assert start == [0, 12, 29, 30, 70] and count == [12, 17, 0, 0, 0] and refused == [2, 3, 4]
    assert t[2] == [7, 5, -1] and t[0] == [4, 3, -1] and free == [] and lens == [17, 0, 17, 0]
    assert pos[:12] == list(range(5, 17)) and slots[0] == 7 * 16 + 5 and slots[11] == 5 * 16
    assert pos[29] == -1 and slots[70] == -1 and pos[71] is None
