"""Pins of the routing oracle: hand-worked scores, selections and groups, and a brute force over all subsets."""
import itertools
import math

import numpy as np
import pytest

from oracle import route as o


def test_scores_by_hand():
    s = o.scores([0.0, math.log(3.0), -math.inf], False)
    assert s == pytest.approx([0.25, 0.75, 0.0], rel=1e-15)
    g = o.scores([0.0, math.log(3.0), -math.inf, -800.0], True)
    assert g[:3] == pytest.approx([0.5, 0.75, 0.0], rel=1e-15) and 0.0 <= g[3] < 1e-300
    assert o.scores([-math.inf, -math.inf], False) == [0.0, 0.0]


def test_selection_by_hand():
    l = [0.0, 1.0, 1.0, -1.0]
    ids, w = o.route_token(l, 2)
    assert ids == [1, 2] and w == [0.5, 0.5]                    # equal logits: the lower index first
    ids, w = o.route_token(l, 2, renormalize=False, scale=2.0)
    z = math.exp(-1) + 2 + math.exp(-2)
    assert w == pytest.approx([2 / z, 2 / z], rel=1e-15)
    # the bias selects and does not weigh
    ids, w = o.route_token(l, 1, bias=[0, 0, 0, 5.0], sigmoid=True, renormalize=False)
    assert ids == [3] and w == pytest.approx([1 / (1 + math.e)], rel=1e-15)


def test_groups_by_hand():
    l = [2.0, -9.0, 1.0, 0.9]                                    # groups {2, -9}, {1, 0.9}
    assert o.route_token(l, 2, n_group=2, topk_group=1, group_top=1, sigmoid=True)[0] == [0, 1]
    assert o.route_token(l, 2, n_group=2, topk_group=1, group_top=2, sigmoid=True)[0] == [2, 3]


def test_unavailable_and_poisoned():
    inf = math.inf
    assert o.route_token([-inf, 0.0, -inf], 2) == ([1, -1], [1.0, 0.0])
    assert o.route_token([-inf] * 3, 2) == ([-1, -1], [0.0, 0.0])
    assert o.route_token([0.0, 1.0], 2, bias=[0.0, -inf], sigmoid=True)[0] == [0, -1]
    for kw in (dict(logits=[math.nan, 0.0]), dict(logits=[inf, 0.0]), dict(logits=[0.0, 0.0], bias=[inf, 0.0])):
        ids, w = o.route_token(kw.pop("logits"), 1, **kw)
        assert ids == [0] and math.isnan(w[0])
    assert o.route_token([inf, 0.0], 1, sigmoid=True) == ([0], [1.0])


def test_brute_force_over_subsets():
    rng = np.random.default_rng(3)
    for _ in range(20):
        l, b = rng.normal(size=7), rng.normal(size=7) * 0.3
        s = 1 / (1 + np.exp(-l))
        best = max(itertools.combinations(range(7), 3), key=lambda c: sum(s[i] + b[i] for i in c))
        ids, w = o.route_token(l, 3, bias=b, sigmoid=True)
        assert sorted(ids) == list(best) and sum(w) == pytest.approx(1.0, rel=1e-14)


def test_group_lists():
    off, order = o.group([[2, 0], [-1, 2], [0, 7]], 3)
    assert off.tolist() == [0, 2, 2, 4] and order.tolist() == [1, 4, 0, 3, 2, 5]
