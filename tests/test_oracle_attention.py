"""Pins of the attention oracle (CPU)."""
from fractions import Fraction

import numpy as np
import pytest
from scipy.special import log_softmax, softmax

from oracle import attention as att


@pytest.mark.parametrize("dim,page", [(64, 32), (96, 64), (128, 128), (256, 32)])
def test_layouts_are_one_to_one(dim, page):
    o, d = np.meshgrid(np.arange(page), np.arange(dim), indexing="ij")
    for index in (att.key_index, att.value_index):
        assert sorted(index(o, d, dim).reshape(-1)) == list(range(page * dim))
    # 8 elements of a key lie together, and 4 places of one value's element
    assert (np.diff(att.key_index(5, np.arange(8), dim)) == 1).all()
    assert (np.diff(att.value_index(np.arange(4, 8), 3, dim)) == 1).all()
    assert att.value_index(8, 3, dim) == att.value_index(0, 3, dim) + 4


def test_turn_by_hand():
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    quarter = np.array([[np.pi / 2, np.pi]])
    assert np.allclose(att.turn(x, quarter, True), [[[-2, 1, -3, -4, 5]]])
    assert np.allclose(att.turn(x, quarter, False), [[[-3, -2, 1, -4, 5]]])


def test_visible_by_hand():
    keys = lambda *a, **k: att.visible(*a, **k)[0].tolist()  # noqa: E731
    assert keys(0, 2, 5) == [0, 1, 2, 3] and keys(1, 2, 5) == [0, 1, 2, 3, 4]
    assert keys(0, 2, 5, window=2) == [2, 3] and keys(0, 2, 5, first=3) == [3]
    assert keys(0, 3, 3, prefix=2) == [0, 1] and keys(0, 3, 3, prefix=9) == [0, 1, 2]
    assert keys(0, 4, 2) == [] and keys(3, 4, 2) == [0, 1]
    # drafted tokens 0 - 1, 0 - 2 over a context of 3; token 3 hangs on the context
    tree = [0b0001, 0b0011, 0b0101, 0b1000]
    k, far = att.visible(2, 4, 7, masks=tree)
    assert k.tolist() == [0, 1, 2, 3, 5] and far.tolist() == [4, 3, 2, 1, 0]
    k, far = att.visible(3, 4, 7, masks=tree, window=3)
    assert k.tolist() == [1, 2, 6] and far.tolist() == [2, 1, 0]
    assert att.visible(1, 2, 3, masks=[1, 0])[0].tolist() == [0]


def test_attend_against_scipy_and_exact():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(3, 4, 8)), rng.normal(size=(7, 2, 8)), rng.normal(size=(7, 2, 8))
    y, lse, dy, dl = att.attend(q, k, v, 3, 7, 0.5, cap=3.0, slopes=np.array([0.1, 0.2, 0.0, 1.0]))
    for i in range(3):
        for h in range(4):
            x = 3 * np.tanh(0.5 * (k[:5 + i, h // 2] @ q[i, h]) / 3)
            x -= [0.1, 0.2, 0.0, 1.0][h] * (4 + i - np.arange(5 + i))
            assert np.allclose(y[i, h], softmax(x) @ v[:5 + i, h // 2], rtol=1e-12)
            assert np.allclose(x - lse[i, h], log_softmax(x), rtol=1e-12)
    assert (dy > 0).all() and (dl > 0).all() and (dl < 1e-4).all()
    # equal scores: the mean of the values
    one = np.zeros((1, 1, 8))
    values = rng.integers(-8, 8, size=(4, 1, 8)).astype(np.float64)
    y, lse, _, _ = att.attend(one, k[:4, :1], values, 1, 4, 1.0)
    assert [Fraction(x).limit_denominator(64) for x in y[0, 0]] == [Fraction(int(s), 4) for s in values.sum(axis=(0, 1))]
    assert np.isclose(lse[0, 0], np.log(4.0))
    # a token that sees nothing
    y, lse, _, _ = att.attend(q[:1], k, v, 1, 7, 1.0, first=[7])
    assert (y == 0).all() and (lse == -np.inf).all()
