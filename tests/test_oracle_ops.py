"""Pins of the oracles of the normalised rotary append, the block-scaled 8-bit
pages and the logits processing: closed forms, library routines, invariants."""
import math

import numpy as np
import pytest
import torch

from oracle import bf16 as OB, bs8_kv as O8, logits as OL, norm_rope as ON, rope as OR


def test_norm_rope_against_complex_products_and_lengths():
    g = np.random.default_rng(0)
    x = g.standard_normal((5, 64)) * 3
    w = g.standard_normal(64)
    y = ON.norm(x, w, 1e-6)
    assert np.allclose((y / w) ** 2 @ np.ones(64), 64.0, rtol=1e-6)
    for pairs in (1, 5, 16, 32):
        for inter in (False, True):
            a = g.uniform(-3, 3, pairs)
            z = ON.rotate(y, np.cos(a), np.sin(a), inter)
            assert np.allclose(np.linalg.norm(z, axis=-1), np.linalg.norm(y, axis=-1))
            assert np.array_equal(z[:, 2 * pairs:], y[:, 2 * pairs:])
            i = np.arange(pairs)
            ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + pairs)
            assert np.allclose(z[:, ia] + 1j * z[:, ib], (y[:, ia] + 1j * y[:, ib]) * np.exp(1j * a))
            assert np.allclose(ON.rotate(z, np.cos(a), -np.sin(a), inter), y)   # and back


def test_norm_rope_half_layout_is_the_plain_rotation():
    cos, sin = OR.table(OR.inv_freq_llama3(), 20)
    x = OB.from_f32_rne(np.random.default_rng(1).standard_normal((3, 64)).astype(np.float32))
    want = OB.to_f64(OR.rotate_bf16(x, cos[19], sin[19]))
    got = ON.rotate(OB.to_f64(x), cos[19], sin[19])
    assert np.abs(got - want).max() <= np.abs(got).max() * 2.0 ** -8


def test_scaled_frequencies():
    plain, mul = ON.inv_freq(32, 10000.0)
    assert mul == 1.0 and np.allclose(plain, OR.inv_freq_plain(10000.0))
    assert np.allclose(ON.inv_freq(32, 10000.0, "linear", 4.0)[0], plain / 4)
    ntk = ON.inv_freq(32, 10000.0, "ntk", 4.0)[0]
    assert ntk[0] == 1.0 and math.isclose(ntk[-1], plain[-1] / 4, rel_tol=1e-12)  # the slowest pair alone is divided whole
    yarn, mul = ON.inv_freq(32, 10000.0, "yarn", 4.0, 4096)
    assert math.isclose(mul, 0.1 * math.log(4.0) + 1)
    turns = 4096 * plain / (2 * math.pi)
    assert np.array_equal(yarn[turns > 40], plain[turns > 40])
    assert np.allclose(yarn[turns < 0.7], plain[turns < 0.7] / 4)
    assert (np.diff(yarn / plain) <= 1e-15).all()


def test_e4m3_codes_are_the_library_types():
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(np.isnan(v), np.isnan(O8.E4M3)) and np.array_equal(v[~np.isnan(v)], O8.E4M3[~np.isnan(v)])
    g = np.random.default_rng(2)
    y = np.concatenate([g.uniform(-470, 470, 4000), g.standard_normal(4000) * 0.02, O8._POS[:-1] + np.diff(O8._POS) / 2,
                        [0.0, -0.0, 448.0, 460.0, -449.0]]).astype(np.float32)
    want = torch.from_numpy(y).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(O8.encode(y, "e4m3"), want)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_block_append_all_at_once_and_token_by_token(kind):
    g = np.random.default_rng(3)
    n = 37
    k = OB.from_f32_rne(g.standard_normal((n, 8, 64)).astype(np.float32))
    v = OB.from_f32_rne((5 * g.standard_normal((n, 8, 64))).astype(np.float32))
    tables = np.array([[2, 0, 3]], np.int32)
    codes0 = g.integers(0, 256, (5, 2, 8, 16, 64)).astype(np.uint8)
    scales0 = np.full((5, 2, 8), np.nan, np.float32)
    codes, scales, _, err = O8.append(codes0, scales0, k, v, [0, n], [n], tables, kind)
    assert not err
    assert np.array_equal(codes[[1, 4]], codes0[[1, 4]])                       # pages of others
    assert np.array_equal(codes[3, :, :, 5:], codes0[3, :, :, 5:])             # slots behind the end
    # int8: half a step of the block's scale, and the quotient's own rounding: it is below 128, so half
    # an fp32 step of it is at most 2^-18.  e4m3: 2^-4 of the value, or half the least step; the
    # quotient's rounding is 2^-24 of the value, 2^-20 of that half step
    for kv, rows in ((0, k), (1, v)):
        x = OB.to_f64(rows)
        for t in range(n):
            page = tables[0, t // 16]
            sc = scales[page, kv].astype(np.float64)[:, None]
            got = O8.decode_codes(codes[page, kv, :, t % 16], kind) * sc
            step = ((0.5 + 2.0 ** -18) * sc if kind == "int8" else
                    (1 + 2.0 ** -20) * np.maximum(2.0 ** -4 * np.abs(x[t]), 2.0 ** -10 * sc))
            assert (np.abs(got - x[t]) <= step).all()
        assert np.allclose(scales[2, kv], np.abs(x[:16]).max((0, 2)) / O8.TOP[kind])
    # token by token: the scales of full blocks end the same, codes within a half step per growth
    c2, s2 = codes0.copy(), scales0.copy()
    for t in range(n):
        c2, s2, _, _ = O8.append(c2, s2, k[t:t + 1], v[t:t + 1], [0, 1], [t + 1], tables, kind)
    assert np.array_equal(s2[[2, 0, 3]], scales[[2, 0, 3]])


def test_block_append_refusals():
    k = np.zeros((3, 8, 64), np.uint16)
    codes, scales = np.full((2, 2, 8, 16, 64), 7, np.uint8), np.ones((2, 2, 8), np.float32)
    for cu, lens, tables in (([0, 3], [2], [[0, 1]]), ([0, 3], [33], [[0, 1]]), ([0, 3], [3], [[2, 1]]),
                             ([0, 4], [4], [[0, 1]]), ([0, 3], [3], [[-1, 1]])):
        c, s, _, err = O8.append(codes, scales, k, k, cu, lens, np.array(tables, np.int32), "int8")
        assert err and np.array_equal(c, codes) and np.array_equal(s, scales)


def test_attend_against_the_library_softmax():
    g = np.random.default_rng(4)
    codes = g.integers(0, 256, (4, 2, 8, 16, 64)).astype(np.uint8)
    scales = g.uniform(0.005, 0.02, (4, 2, 8)).astype(np.float32)
    tables, lens = np.array([[3, 1, -1], [0, 2, -1]], np.int32), [32, 21]
    q = OB.from_f32_rne(g.standard_normal((2, 32, 64)).astype(np.float32))
    out, size, _, _ = O8.attend(q, codes, scales, tables, lens, 0.125, "int8")
    for s in range(2):
        kv = torch.from_numpy(O8.values(codes[tables[s, :2]], scales[tables[s, :2]], "int8"))
        kv = kv.permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, :lens[s]].repeat_interleave(4, 1)
        want = torch.nn.functional.scaled_dot_product_attention(
            torch.from_numpy(OB.to_f64(q[s]))[:, None], kv[0], kv[1], scale=0.125)[:, 0].numpy()
        assert np.abs(out[s] - want).max() < 1e-12
    assert (size >= np.abs(out) - 1e-15).all()


def test_logits_worked_example():
    x = np.array([[2.0, -1.0, 0.5, 3.0, 0.0]], np.float32)
    hist = np.array([[0, 1, 3, 3, -1, 9]], np.int32)
    out, ids = OL.process(x, hist, [6], [1], [2.0], [0.25], [0.5], np.array([[2, 2, -1]]),
                          np.array([[9.0, 1.0, 5.0]], np.float32), None)
    # 0: prompt only: 2 / 2; 1: -1 * 2 - .5 - .25; 3: 3 / 2 - 2 * .5 - .25; 2: last bias; 4: untouched
    assert np.array_equal(out, np.array([[1.0, -2.75, 1.5, 0.25, 0.0]], np.float32)) and ids[0] == 2
    out, ids = OL.process(x, mask=np.array([[0b10010]], np.int32))
    assert np.array_equal(out[0], np.array([-np.inf, -1, -np.inf, -np.inf, 0], np.float32)) and ids[0] == 4
    _, ids = OL.process(np.array([[np.nan, 1.0], [np.nan, np.nan], [1.0, 1.0]], np.float32),
                        mask=np.array([[1], [3], [0]], np.int32))
    assert ids.tolist() == [-1, -1, -1]
    _, ids = OL.process(np.array([[-np.inf, -np.inf]], np.float32))
    assert ids[0] == 0                                                      # allowed, and the largest
