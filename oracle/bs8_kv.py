"""Block-scaled 8-bit K/V pages (test infrastructure only).

A block is the 16 slots of one page, K or V, and KV head; it has one fp32
scale.  Codes are int8 or e4m3 (1 sign, 4 exponent bits of bias 7, 3 mantissa
bits, no infinities, largest 448):
    scale = fp32(amax / top),  code = nearest-even(fp32(x / scale)),
top = 127 (clamped to [-127, 127]) or 448 (saturating); scale 0 gives code 0.
The new tokens of a call that fall into one block set its scale together:
anew from slot 0 on, else the larger of the scale found and theirs; when that
grows, a held code becomes the code of fp32(fp32(code * old) / new).

Rows are finite here.

Arrays: codes uint8 bytes [pages][2][8][16][64], scales float32 [pages][2][8].
fp32 divisions and products are FP64 ones rounded once, which is the same.
"""
from __future__ import annotations

import numpy as np

from . import bf16, rope
from .paged_kv import GROUP, HEAD_DIM, NUM_KV_HEADS, NUM_Q_HEADS, PAGE_TOKENS

TOP = {"int8": 127.0, "e4m3": 448.0}


def _e4m3_values():
    v = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = (m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
        v[b] = np.nan if (b & 0x7F) == 0x7F else (-x if b & 0x80 else x)
    return v


E4M3 = _e4m3_values()
_POS = E4M3[:127]  # 0 .. 448, ascending; byte b is its index


def encode(y, kind):
    """Bytes of fp32 quotients y."""
    y = np.asarray(y, np.float64)
    if kind == "int8":
        return np.clip(np.rint(y), -127, 127).astype(np.int8).view(np.uint8)
    mag = np.minimum(np.abs(y), 448.0)
    hi = np.clip(np.searchsorted(_POS, mag), 0, 126)      # first value >= mag
    lo = np.maximum(hi - 1, 0)
    dh, dl = _POS[hi] - mag, mag - _POS[lo]
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))          # ties to the even mantissa
    b = np.where(_POS[hi] == mag, hi, np.where(up, hi, lo)).astype(np.uint8)
    return np.where(np.signbit(y), b | 0x80, b).astype(np.uint8)


def decode_codes(b, kind):
    b = np.asarray(b, np.uint8)
    return b.view(np.int8).astype(np.float64) if kind == "int8" else E4M3[b]


def _f32(x):
    return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


def quantise(x, scale, kind):
    if scale == 0:
        return np.zeros(np.shape(x), np.uint8)
    return encode(_f32(np.asarray(x, np.float64) / np.float64(scale)), kind)


def append(codes, scales, k_bits, v_bits, cu, lens, tables, kind, cos=None, sin=None, q_bits=None):
    """One call on copies: (codes, scales, rotated q bits or None, error seen).
    Rows the library leaves untouched are 0 in the returned q."""
    codes, scales = codes.copy(), scales.copy()
    q_out = None if q_bits is None else np.zeros_like(q_bits)
    T, (S, M), pages = k_bits.shape[0], tables.shape, codes.shape[0]
    err = False
    for s in range(len(lens)):
        lo, hi, n = int(cu[s]), int(cu[s + 1]), int(lens[s])
        if hi <= lo:
            continue
        if hi > T or n < hi - lo or n > M * PAGE_TOKENS or (cos is not None and n > cos.shape[0]):
            err = True
            continue
        pos = n - (hi - lo)
        t = lo
        while t < hi:
            slot = pos % PAGE_TOKENS
            m = min(PAGE_TOKENS - slot, hi - t)
            page = int(tables[s, pos // PAGE_TOKENS])
            if not 0 <= page < pages:
                err = True
            else:
                kr = k_bits[t:t + m]
                if cos is not None:
                    kr = np.stack([rope.rotate_bf16(kr[i], cos[pos + i], sin[pos + i]) for i in range(m)])
                    if q_bits is not None:
                        for i in range(m):
                            q_out[t + i] = rope.rotate_bf16(q_bits[t + i], cos[pos + i], sin[pos + i])
                for kv, rows in ((0, bf16.to_f64(kr)), (1, bf16.to_f64(v_bits[t:t + m]))):
                    for g in range(NUM_KV_HEADS):
                        x = rows[:, g]
                        fresh = np.float32(np.abs(x).max() / TOP[kind])
                        old = scales[page, kv, g]
                        now = fresh if slot == 0 or fresh > old else old
                        if slot and fresh > old:
                            held = _f32(decode_codes(codes[page, kv, g, :slot], kind) * np.float64(old))
                            codes[page, kv, g, :slot] = quantise(held, now, kind)
                        codes[page, kv, g, slot:slot + m] = quantise(x, now, kind)
                        scales[page, kv, g] = now
            t, pos = t + m, pos + m
    return codes, scales, q_out, err


def values(codes, scales, kind):
    return decode_codes(codes, kind) * scales.astype(np.float64)[..., None, None]


def attend(q_bits, codes, scales, tables, lens, scale, kind):
    """FP64 attention and the sizes its error bounds are made of: (out, sum of
    p |v| over sum of p, the largest |scale| sum |q| |k| of each head, the
    largest |v| of each head)."""
    S = len(lens)
    out = np.zeros((S, NUM_Q_HEADS, HEAD_DIM))
    size, reach, most = np.zeros_like(out), np.zeros((S, NUM_Q_HEADS, 1)), np.zeros((S, NUM_Q_HEADS, 1))
    q = bf16.to_f64(q_bits)
    for s in range(S):
        n = int(lens[s])
        if n <= 0 or n > tables.shape[1] * PAGE_TOKENS:
            continue
        ids = tables[s, :-(-n // PAGE_TOKENS)]
        if (ids < 0).any() or (ids >= codes.shape[0]).any():
            continue
        kv = values(codes[ids], scales[ids], kind)
        kv = kv.transpose(1, 2, 0, 3, 4).reshape(2, NUM_KV_HEADS, -1, HEAD_DIM)[:, :, :n]
        for h in range(NUM_Q_HEADS):
            k, v = kv[0, h // GROUP], kv[1, h // GROUP]
            x = scale * (k @ q[s, h])
            p = np.exp(x - x.max())
            out[s, h] = p @ v / p.sum()
            size[s, h] = p @ np.abs(v) / p.sum()
            reach[s, h] = abs(scale) * (np.abs(k) @ np.abs(q[s, h])).max()
            most[s, h] = np.abs(v).max()
    return out, size, reach, most
