"""Pins of the 4-bit pages' oracle: the block's layout, the codes of a row against
brute force, attention against the bf16 oracle."""
import re
import os

import numpy as np
import pytest

from oracle import bf16 as OB, int4_kv as O4, paged_kv as OP

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_half_byte_has_one_place():
    used = np.zeros((O4.BLOCK_BYTES, 2), int)
    for kv in range(2):
        for r in range(16):
            for d in range(64):
                used[O4.CODE_AT[kv, r, d], d % 2] += 1
            used[O4.SCALE_AT[kv, r]:O4.SCALE_AT[kv, r] + 4] += 1
    assert (used == 1).all()
    text = open(os.path.join(ROOT, "include", "pkv.h")).read()
    assert int(re.search(r"#define PKV_I4_BLOCK_BYTES (\d+)", text).group(1)) == O4.BLOCK_BYTES


@pytest.mark.parametrize("size", [1.0, 1e-30, 1e30, 3e38])
def test_codes_are_the_nearest(size):
    g = np.random.default_rng(1)
    x = OB.from_f32_rne((np.clip(g.standard_normal((50, 64)), -1.1, 1.1) * size / 1.1).astype(np.float32))
    codes, scale, lo = O4.quantise(x)
    v, s, m = OB.to_f64(x), OB.to_f64(scale)[:, None], OB.to_f64(lo)[:, None]
    assert np.array_equal(m[:, 0], v.min(1))
    # half a step, and the top of a row whose scale was rounded down: 15 * 2^-9 steps
    assert (np.abs(m + codes * s - v) <= s * (0.5 + 1e-6)).all()
    assert (np.abs((v.max(1) - v.min(1)) / 15 / s[:, 0] - 1) <= 2.0 ** -8 * (1 + 1e-6)).all()
    ends = np.sort(codes, 1)
    assert (ends[:, 0] == 0).all() and (ends[:, -1] == 15).all()


def test_flat_tiny_and_not_finite_rows():
    x = np.zeros((6, 64), np.uint16)
    x[0] = OB.from_f32_rne(np.float32(-3.5))
    x[1, 3], x[1, 5] = 1, 0x8001                    # subnormal
    x[2, 7] = 0x8000                                # a -0 among zeros
    x[3, 1] = 0x7F80
    x[4, 1] = 0x7FC1
    x[5, 0] = 0xFF80
    codes, scale, lo = O4.quantise(x)
    assert not codes.any() and (scale[:3] == 0).all() and (scale[3:] == O4.NAN).all() and (lo[3:] == O4.NAN).all()
    assert lo[0] == x[0, 0] and lo[1] == 0x8001 and lo[2] == 0x8000


def test_append_and_attention():
    g = np.random.default_rng(2)
    k, v, q = (OB.from_f32_rne(g.standard_normal((n, h, 64)).astype(np.float32)) for n, h in ((21, 8), (21, 8), (1, 32)))
    bt = np.array([[2, 0]], np.int32)
    pool, _, err = O4.append(O4.new_pool(3), k, v, [0, 21], [21], bt)
    assert not err
    x = O4.values(pool)
    for t in range(21):
        for kv, rows in ((0, k), (1, v)):
            got, want = x[bt[0, t // 16], kv, :, t % 16], OB.to_f64(rows[t])
            step = (want.max(-1) - want.min(-1))[:, None] / 15
            assert (np.abs(got - want) <= step * (0.5 + 2.0 ** -7)).all()
    out = O4.attend(q, pool, bt, [21], 0.125)[0]
    wide = OB.from_f64_via_f32(x)                   # the values rounded to bf16
    ref, _ = OP.decode(q, wide, bt, [21], 0.125)
    assert np.abs(out - ref).max() < 2e-2
    assert O4.append(O4.new_pool(3), k, v, [0, 21], [20], bt)[2] and O4.append(O4.new_pool(2), k, v, [0, 21], [21], bt)[2]
