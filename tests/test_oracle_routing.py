"""Pins of the routing and adapter oracle (CPU)."""
import itertools
from fractions import Fraction

import numpy as np
import pytest
from scipy.special import expit, softmax

from oracle import routing

NAN, INF = float("nan"), float("inf")


def test_route_by_hand():
    # three of five, softmax, no bias: the order of the logits, ties to the lower index
    e, w = routing.route(np.array([[1.0, 3.0, 3.0, -INF, 2.0]]), 3)
    assert e.tolist() == [[1, 2, 4]]
    p = np.exp([3.0, 3.0, 2.0])
    assert np.allclose(w, p / p.sum(), rtol=1e-15)
    # a bias moves the choice, not the weight
    e, w = routing.route(np.array([[0.0, 0.0, 0.0]]), 1, score=routing.SIGMOID, bias=[0.0, 0.5, -INF], renormalise=False,
                         scale=2.0)
    assert e.tolist() == [[1]] and w.tolist() == [[1.0]]
    # nothing left: -1 and 0
    e, w = routing.route(np.array([[-INF, NAN], [5.0, -INF]]), 2)
    assert e.tolist() == [[-1, -1], [0, -1]] and w.tolist() == [[0.0, 0.0], [1.0, 0.0]]
    # +inf is the largest finite value: two of them share
    e, w = routing.route(np.array([[INF, 1.0, INF]]), 2, renormalise=False)
    assert e.tolist() == [[0, 2]] and w.tolist() == [[0.5, 0.5]]


def test_route_groups_by_hand():
    l = np.array([[9.0, 0.0, 0.0, 0.0, 5.0, 5.0]])
    e, _ = routing.route(l, 2, score=routing.SIGMOID, groups=3, top_groups=1)
    assert e.tolist() == [[0, 1]]  # the group of the largest logit
    e, _ = routing.route(l, 2, score=routing.SIGMOID, groups=3, top_groups=1, group_score=routing.GROUP_TOP2)
    assert e.tolist() == [[4, 5]]  # 2 sigmoid(5) > sigmoid(9) + sigmoid(0)


@pytest.mark.parametrize("score", [routing.SOFTMAX, routing.SIGMOID])
@pytest.mark.parametrize("pairs", [routing.GROUP_MAX, routing.GROUP_TOP2])
def test_route_by_brute_force(score, pairs):
    rng = np.random.default_rng(3)
    l, b = rng.normal(size=(20, 12)), rng.normal(size=12) * 0.2
    s = softmax(l, axis=1) if score == routing.SOFTMAX else expit(l)
    e, w = routing.route(l, 3, score, b, groups=4, top_groups=2, group_score=pairs, renormalise=False)
    for t in range(20):
        c = s[t] + b
        best = lambda g: sum(sorted(c[3 * g:3 * g + 3])[-1 - pairs:])  # noqa: E731
        kept = max(itertools.combinations(range(4), 2), key=lambda gs: sum(map(best, gs)))
        inside = [i for i in range(12) if i // 3 in kept]
        want = max(itertools.combinations(inside, 3), key=lambda es: sum(c[list(es)]))
        assert set(e[t]) == set(want)
        assert list(c[e[t]]) == sorted(c[e[t]], reverse=True)
        assert np.allclose(w[t], s[t][e[t]], rtol=1e-13)


def test_rows_by_hand():
    offsets, order, slot = routing.group_rows(np.array([[2, 0], [-1, 2], [0, 7]]), 3)
    assert offsets.tolist() == [0, 2, 2, 4]
    assert order.tolist() == [1, 4, 0, 3, 2, 5]
    assert slot.tolist() == [[2, 0], [-1, 3], [1, -1]]
    x = np.array([[1.0], [2.0], [3.0]])
    xs = routing.dispatch_rows(x, slot, np.full((6, 1), 9.0))
    assert xs[:, 0].tolist() == [1, 3, 1, 2, 9, 9]
    y, size = routing.combine_rows(xs, slot, np.array([[1.0, 2.0], [5.0, -1.0], [1.0, 1.0]]), np.full((3, 1), 10.0))
    assert y[:, 0].tolist() == [13, 8, 13] and size[:, 0].tolist() == [13, 12, 13]


def test_lora_is_the_merged_weight():
    rng = np.random.default_rng(5)
    x = rng.integers(-8, 8, size=(3, 6)).astype(np.float64)
    w = rng.integers(-4, 4, size=(4, 6)).astype(np.float64)
    a, b = rng.integers(-4, 4, size=(2, 6)).astype(np.float64), rng.integers(-4, 4, size=(4, 2)).astype(np.float64)
    y = routing.lora(x, [1, -1, 1], {1: (a, b, 0.5)}, x @ w.T)
    for t in range(3):
        for n in range(4):
            m = [Fraction(w[n, k]) + (Fraction(1, 2) * sum(Fraction(b[n, r]) * Fraction(a[r, k]) for r in range(2))
                                      if t != 1 else 0) for k in range(6)]
            assert Fraction(y[t, n]) == sum(Fraction(x[t, k]) * m[k] for k in range(6))
    assert (routing.lora_error_bound(x, [1, -1, 1], {1: (a, b, 0.5)}, x @ w.T) > 0).any()
