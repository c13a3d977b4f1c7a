"""The sampler's oracle, pinned by hand cases and by frequencies."""
import math

import numpy as np
import pytest

from oracle import sampling as s

ROW = np.log(np.array([0.1, 0.4, 0.05, 0.25, 0.2], np.float64))


def test_filters_by_hand():
    assert s.kept(ROW).tolist() == [0, 1, 2, 3, 4]
    assert s.kept(ROW, top_k=2).tolist() == [1, 3]
    assert s.kept(ROW, top_p=0.6).tolist() == [1, 3]               # 0.4 < 0.6, 0.65 is enough
    assert s.kept(ROW, top_p=0.7).tolist() == [1, 3, 4]
    assert s.kept(ROW, top_k=3, top_p=0.7).tolist() == [1, 3]      # of 0.85: 0.595
    assert s.kept(ROW, min_p=0.3).tolist() == [1, 3, 4]
    assert s.kept(ROW, top_p=0.0).tolist() == [1]
    assert s.kept(ROW, temperature=0.0, top_k=3).tolist() == [1]
    assert s.kept(ROW, min_p=2.0).tolist() == [1]
    assert s.kept(np.array([1.0, np.nan, 3.0, -np.inf, 3.0]), top_k=2).tolist() == [2, 4]
    assert s.kept(np.array([1.0, 3.0, 3.0, 3.0]), top_k=2).tolist() == [1, 2]
    assert s.kept(np.full(4, -np.inf)).tolist() == []
    assert s.kept(np.array([0.0, np.inf, 1.0, np.inf]), top_p=0.9).tolist() == [1, 3]


def test_draws_by_hand():
    every = s.kept(ROW)
    for u, token in ((0.0, 0), (0.0999, 0), (0.1001, 1), (0.4999, 1), (0.5001, 2), (0.5499, 2), (0.56, 3), (0.81, 4),
                     (0.99999, 4), (1.0, 4), (-1.0, 0), (math.nan, 0)):
        assert s.draw(ROW, every, 1.0, u)[0] == token, u
    assert s.draw(ROW, every, 1.0, 0.3)[1] == pytest.approx(0.4)
    assert s.draw(ROW, every, 1.0, 0.3, without=1) == (3, pytest.approx(0.25 / 0.6))
    assert s.draw(ROW, np.array([1]), 1.0, 0.3, without=1) == (-1, 0.0)
    assert s.draw(ROW, np.array([1, 3]), 0.5, 0.8)[1] == pytest.approx(0.0625 / 0.2225)
    assert s.p_draft(ROW, np.array([1, 3]), 1.0, 3) == pytest.approx(0.25 / 0.65)
    assert s.p_draft(ROW, np.array([1, 3]), 1.0, 2) == 0.0


def test_frequencies():
    n = 20000
    got = np.bincount([s.draw(ROW, np.arange(5), 1.0, (i + 0.5) / n)[0] for i in range(n)], minlength=5) / n
    assert np.all(np.abs(got - np.exp(ROW)) <= 1.0 / n)


def test_accepting_and_drawing_another_gives_the_distribution():
    """P(draft d accepted) + P(refused) * P(other) is the distribution itself."""
    every = np.arange(5)
    for d in range(5):
        p = s.p_draft(ROW, every, 1.0, d)
        n = 4000
        other = np.bincount([s.draw(ROW, every, 1.0, (i + 0.5) / n, without=d)[0] for i in range(n)], minlength=5) / n
        whole = (1 - p) * other
        whole[d] += p
        assert np.all(np.abs(whole - np.exp(ROW)) <= 2.0 / n)
