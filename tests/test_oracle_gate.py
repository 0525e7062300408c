"""Pins of the gated-routing oracle: hand-worked choices and weights, and a
brute-force choice over every subset."""
import itertools
import math
import random

import pytest

from oracle import gate

LOW = -3.4028234663852886e38


def test_hand_worked_softmax_and_sigmoid():
    ids, w = gate.token([0.0, math.log(2.0), -math.inf, math.log(4.0)], LOW, 2)
    assert ids == [3, 1] and w == pytest.approx([4 / 7, 2 / 7])
    ids, w = gate.token([0.0, math.log(3.0), 0.0], LOW, 2, score="sigmoid", renorm=True, scale=2.0)
    assert ids == [1, 0]
    assert w == pytest.approx([2 * 0.75 / 1.25, 2 * 0.5 / 1.25])


def test_bias_counts_in_the_choice_only():
    ids, w = gate.token([0.0, 2.0, 1.0], LOW, 1, score="sigmoid", bias=[5.0, 0.0, 0.0])
    assert ids == [0] and w == [0.5]
    # a bias of -inf takes an expert out
    ids, _ = gate.token([0.0, 2.0, 1.0], LOW, 3, score="sigmoid", bias=[0.0, -math.inf, 0.0])
    assert ids == [2, 0, -1]


def test_groups_ties_and_what_is_not_to_be_had():
    # groups {0, 1}, {2, 3}, {4, 5}: largest 3, 3, 2; sums differ
    l = [3.0, -9.0, 3.0, 2.0, 2.0, 2.0]
    assert gate.token(l, LOW, 2, n_group=3, topk_group=1)[0] == [0, 1]
    assert gate.token(l, LOW, 2, score="sigmoid", n_group=3, topk_group=1, top2=True)[0] == [2, 3]
    assert gate.token([1.0, 1.0, 1.0], LOW, 2)[0] == [0, 1]
    assert gate.token([math.nan, LOW, -math.inf, 1.0], LOW, 2) == ([3, -1], [1.0, 0.0])
    assert gate.token([1.0, 2.0], LOW, 2, live=False) == ([-1, -1], [0.0, 0.0])


def test_renormalised_weights_survive_underflow():
    ids, w = gate.token([-2000.0, -2001.0], LOW, 2, score="sigmoid", renorm=True)
    assert ids == [0, 1] and w == pytest.approx([1 / (1 + math.exp(-1)), 1 / (1 + math.exp(1))])
    ids, w = gate.token([math.inf, math.inf, 0.0], LOW, 3)
    assert ids == [0, 1, 2] and w == [0.5, 0.5, 0.0]


def test_choice_is_the_best_subset():
    rng = random.Random(3)
    for _ in range(100):
        E, k = 6, rng.randint(1, 4)
        l = [rng.gauss(0, 1) for _ in range(E)]
        b = [rng.gauss(0, 0.3) for _ in range(E)]
        ids, _ = gate.token(l, LOW, k, score="sigmoid", bias=b)
        c = [1 / (1 + math.exp(-v)) + u for v, u in zip(l, b)]
        best = max(itertools.combinations(range(E), k), key=lambda s: sum(c[e] for e in s))
        assert sorted(ids) == sorted(best)
        assert [c[e] for e in ids] == sorted((c[e] for e in ids), reverse=True)
