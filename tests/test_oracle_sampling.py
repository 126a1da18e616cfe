"""Pins of the sampler's oracle: the limits by brute force, the race's distribution."""
import numpy as np
import pytest

from oracle import sampling as S


@pytest.mark.parametrize("k,p,floor", [(0, 1.0, 0.0), (3, 1.0, 0.0), (0, 0.5, 0.0), (0, 1.0, 0.3), (4, 0.6, 0.1), (1, 0.9, 0.0),
                                       (0, 0.0, 0.0), (0, 1.0, 2.0)])
def test_limits_by_brute_force(k, p, floor):
    g = np.random.default_rng(1)
    for _ in range(20):
        x = np.round(g.normal(0, 1.5, 12), 1)      # with ties
        T = g.uniform(0.3, 2)
        order, n, lp = S.limits(x, T, k, p, floor)
        w = np.exp((x - x.max()) / T)
        for i in range(12):
            front = [j for j in range(12) if x[j] > x[i] or (x[j] == x[i] and j < i)]
            ok = not front or ((k == 0 or len(front) < k) and (p >= 1 or w[front].sum() < p * w.sum()) and w[i] >= floor)
            assert ok == (i in order[:n])
        assert np.allclose(np.exp(lp), w / w.sum())


def test_race_follows_the_distribution():
    g = np.random.default_rng(2)
    x, T = np.array([1.0, 0.0, 2.0, -1.0, 1.5]), 0.8
    got = np.bincount([S.sample(x, g.exponential(size=5), T, k=4)[0] for _ in range(20000)], minlength=5)
    w = np.exp(x / T) * [1, 1, 1, 0, 1]
    q = w / w.sum()
    assert (np.abs(got - 20000 * q) <= 5 * np.sqrt(20000 * q * (1 - q)) + 1e-9).all()


def test_special_rows():
    assert S.sample([-np.inf, np.nan], [1, 1]) [0] == -1
    assert S.sample([1.0, 2.0], [1, 1], T=-1.0)[0] == S.sample([1.0, 2.0], [1, 1], p=np.nan)[0] == -1
    assert S.sample([3.0, np.nan, 3.0], [9, 9, 1e-9], T=0)[0] == 0
    assert S.sample([np.inf, 5.0, np.inf], [2, 1e-30, 1])[0] == 2
    assert S.sample([1.0, 1.0, 1.0], [3, 2, 1], k=2)[0] == 1     # ties: the lowest ids are kept
    assert S.acceptable(1, [1.0, 1.0, 0.0], [1 + 1e-6, 1, 5]) and not S.acceptable(2, [1.0, 1.0, 0.0], [1, 1, 5])
