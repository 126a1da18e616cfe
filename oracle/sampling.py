"""The next token from softmax(logits / T) restricted by top-k, top-p and min-p, by
the race of given exponential variates (test infrastructure only), in FP64 with a
sort, as the definition reads.

limits() also gives the sets that are kept when every bound is moved by a relative
`slack` against or for the token: what a computation in 32 bits may decide either way
lies between them.
"""
from __future__ import annotations

import numpy as np

LARGEST = float(np.finfo(np.float32).max)


def _tamed(x):
    """NaN as -inf, +inf as the largest number."""
    x = np.asarray(x, np.float64)
    return np.minimum(np.where(np.isnan(x), -np.inf, x), LARGEST)


def limits(x, T, k=0, p=1.0, floor=0.0, slack=0.0):
    """(order by rank, how many of it are kept, log-probabilities) of one row."""
    x = _tamed(x)
    with np.errstate(all="ignore"):
        y = (x - x.max()) / T
        w = np.exp(y)
    order = np.argsort(-x, kind="stable")
    z = w.sum()
    before = np.concatenate([[0.0], np.cumsum(w[order])[:-1]])
    keep = np.isfinite(x[order])
    if 0 < k < len(x):
        keep &= np.arange(len(x)) < k
    if p < 1:
        keep &= before < p * z * (1 + slack)
    if floor > 0:
        keep &= w[order] >= floor * (1 - slack)
    keep[0] = True
    n = int(np.argmin(keep)) if not keep.all() else len(x)
    assert not keep[n:].any()                      # a prefix
    return order, n, y - np.log(z)


def race(x, noise, T):
    """log(w / noise)."""
    x = _tamed(x)
    e = np.asarray(noise, np.float64)
    e = np.minimum(np.where(np.isnan(e) | (e < 2.0 ** -126), 2.0 ** -126, e), LARGEST)
    with np.errstate(all="ignore"):
        return (x - x.max()) / T - np.log(e)


def sample(x, noise, T=1.0, k=0, p=1.0, floor=0.0):
    """(id, log-probability) of one row."""
    x = _tamed(x)
    if not (0 <= T < np.inf) or np.isnan(p) or np.isnan(floor) or not (x > -np.inf).any():
        return -1, np.nan
    if T == 0:
        order, _, lp = limits(x, 1.0)
        return int(order[0]), float(lp[order[0]])
    order, n, lp = limits(x, T, k, p, floor)
    r = race(x, noise, T)
    best = min(order[:n], key=lambda i: (-r[i], i))
    return int(best), float(lp[best])


def acceptable(got, x, noise, T=1.0, k=0, p=1.0, floor=0.0, slack=2e-5):
    """Whether 32 bits may give this id: kept under the moved limits, and at most
    `slack` behind the best that is kept whatever the rounding."""
    want, _ = sample(x, noise, T, k, p, floor)
    if got == want:
        return True
    if got < 0 or want < 0 or T == 0:
        return False
    r = race(x, noise, T)
    order, most, _ = limits(x, T, k, p, floor, slack)
    _, least, _ = limits(x, T, k, p, floor, -slack)
    return got in order[:most] and r[got] >= r[order[:least]].max() - slack
