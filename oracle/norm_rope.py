"""Per-head RMS norm and rotation of q and k (test infrastructure only).

For a head row x of 64 values, weights w (or none) and the first 2 P dims
rotated by one position's table row (P pairs):
    y = x / sqrt(mean(x^2) + eps) * w         (y = x without w)
    pairs (i, i + P), or (2 i, 2 i + 1) when interleaved:
    (a, b) -> (a c_i - b s_i, a s_i + b c_i); the other dims unchanged.
Everything in FP64, nothing rounded: the library's result is this value
rounded to bf16 once, up to fp32 arithmetic.

Also the frequencies of a rotary dimension and their scalings for long
contexts (linear interpolation, enlarged base, and the ramp between the two
over the pairs: kept above `beta_fast` turns of the original context, divided
below `beta_slow`).
"""
from __future__ import annotations

import math

import numpy as np

HEAD_DIM = 64


def norm(x, w, eps):
    x = np.asarray(x, np.float64)
    if w is None:
        return x
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * np.asarray(w, np.float64)


def rotate(y, cos_row, sin_row, interleaved=False):
    """Rotate [..., 64] by table rows broadcast against [..., P]."""
    c, s = np.asarray(cos_row, np.float64), np.asarray(sin_row, np.float64)
    p = c.shape[-1]
    out = np.array(y, np.float64)
    ia, ib = (np.arange(p) * 2, np.arange(p) * 2 + 1) if interleaved else (np.arange(p), np.arange(p) + p)
    a, b = out[..., ia].copy(), out[..., ib].copy()
    out[..., ia] = a * c - b * s
    out[..., ib] = a * s + b * c
    return out


def pair_sizes(y, pairs, interleaved=False):
    """|a| + |b| of each dim's pair (|y| for a dim outside the rotation): the
    scale of the rotation's rounding errors."""
    m = np.abs(np.asarray(y, np.float64))
    i = np.arange(pairs)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
    both = m[..., ia] + m[..., ib]
    m[..., ia] = both
    m[..., ib] = both
    return m


def inv_freq(pairs, theta, scaling=None, factor=1.0, original_max_pos=8192, beta_fast=32.0, beta_slow=1.0):
    """(inv_freq [pairs], attention factor), pair by pair."""
    d, mul = 2 * pairs, 1.0
    if scaling == "ntk":
        theta = theta * factor ** (d / (d - 2))
    out = []
    for i in range(pairs):
        f = theta ** (-2.0 * i / d)
        if scaling == "linear":
            f = f / factor
        elif scaling == "yarn":
            def at(turns):
                return pairs * math.log(original_max_pos / (turns * 2 * math.pi)) / math.log(theta)
            lo, hi = max(0, math.floor(at(beta_fast))), min(d - 1, math.ceil(at(beta_slow)))
            r = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f = f / factor * r + f * (1.0 - r)
            mul = 0.1 * math.log(factor) + 1.0
        out.append(f)
    return np.array(out), mul
