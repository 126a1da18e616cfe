"""4-bit K/V pages (test infrastructure only).

Every row (token, KV head, K or V) of 64 values has a scale, a minimum and codes
of 4 bits.  With lo and hi the smallest and largest value of the row, in fp32:
    scale = bf16((hi / 2 - lo / 2) / 7.5), 0 where that is below 2^-126
    inv   = 2 / scale
    code  = nearest-even((x / 2 - lo / 2) * inv)
and a code c stands for lo + c * scale.  A row that is not finite has scale = lo =
NaN and codes 0.  lo is -0 if the least value is a zero and one of them is -0.

Pool: uint8 [pages][8 heads][1152]; positions() says where a block keeps what.
fp32 operations are FP64 ones rounded once, which is the same here (sums of two
bf16 values that need more than 53 bits round to the larger one either way).
"""
from __future__ import annotations

import numpy as np

from . import bf16, rope
from .paged_kv import GROUP, HEAD_DIM, NUM_KV_HEADS, NUM_Q_HEADS, PAGE_TOKENS

BLOCK_BYTES = 1152
NAN = 0x7FC0


def positions():
    """(byte of the code of [K|V][slot][dim], even dims in its low half; byte of the
    scale of [K|V][slot], the minimum 2 behind it)."""
    code = np.zeros((2, PAGE_TOKENS, HEAD_DIM), np.int64)
    scale = np.zeros((2, PAGE_TOKENS), np.int64)
    for r in range(PAGE_TOKENS):
        u, g = divmod(r, 8)
        for d in range(HEAD_DIM):
            code[0, r, d] = 16 * (4 * g + d // 16) + 8 * u + d % 16 // 2
            code[1, r, d] = 512 + 16 * (4 * (d // 8) + g // 2) + 8 * u + 4 * (d % 8 // 4) + 2 * (g % 2) + d % 4 // 2
        scale[:, r] = 1024 + 16 * g + 4 * u, 1024 + 16 * g + 4 * u + 8
    return code, scale


CODE_AT, SCALE_AT = positions()
EVEN = np.arange(HEAD_DIM) % 2 == 0


def new_pool(pages):
    return np.zeros((pages, NUM_KV_HEADS, BLOCK_BYTES), np.uint8)


def quantise(x_bits):
    """(codes uint8 [..., 64], scale bits, minimum bits) of rows of bf16 bits [..., 64]."""
    x = bf16.to_f64(x_bits)
    f32 = np.float32
    finite = np.isfinite(x).all(-1)
    safe = np.where(finite[..., None], x, 0.0)
    lo, hi = safe.min(-1), safe.max(-1)
    minus = (lo == 0) & ((np.asarray(x_bits) == 0x8000).any(-1))
    with np.errstate(all="ignore"):
        half = f32(hi / 2 - lo / 2).astype(f32)
        s = bf16.from_f32_rne(f32(half.astype(np.float64) / 7.5))
        s = np.where(bf16.to_f64(s) < 2.0 ** -126, 0, s).astype(np.uint16)
        sv = bf16.to_f64(s)
        inv = np.where(sv > 0, (2.0 / np.where(sv > 0, sv, 1.0)).astype(f32), f32(0)).astype(np.float64)
        y = f32(safe / 2 - (lo / 2)[..., None]).astype(np.float64) * inv[..., None]
        codes = np.rint(y.astype(f32)).astype(np.int64)
    assert codes.min() >= 0 and codes.max() <= 15
    lo_bits = bf16.from_f32_rne(lo.astype(f32))
    lo_bits = np.where(minus, 0x8000, np.where(lo == 0, 0, lo_bits))
    return (codes.astype(np.uint8), np.where(finite, s, NAN).astype(np.uint16), np.where(finite, lo_bits, NAN).astype(np.uint16))


def write_row(block, kv, slot, codes, scale, lo):
    """One row into a block (bytes [1152])."""
    for d in range(0, HEAD_DIM, 2):
        block[CODE_AT[kv, slot, d]] = int(codes[d]) | int(codes[d + 1]) << 4
    at = SCALE_AT[kv, slot]
    block[at:at + 4] = np.array([scale, lo], np.uint16).view(np.uint8)


def codes_of(pool):
    """(codes [..., 2, 16, 64], scales, minima [..., 2, 16] as float64) of blocks [..., 1152]."""
    pool = np.asarray(pool)
    b = pool[..., CODE_AT]
    both = np.stack([pool[..., SCALE_AT + i].astype(np.uint16) for i in range(4)], -1)
    scale, lo = both[..., 0] | both[..., 1] << 8, both[..., 2] | both[..., 3] << 8
    return np.where(EVEN, b & 15, b >> 4), bf16.to_f64(scale), bf16.to_f64(lo)


def values(pool):
    """The values of pages [n][8][1152] as [n][2][8][16][64]."""
    c, s, lo = codes_of(pool)
    return (lo[..., None] + c * s[..., None]).swapaxes(1, 2)


def append(pool, k_bits, v_bits, cu, lens, tables, cos=None, sin=None, q_bits=None):
    """One call on copies: (pool, rotated q bits or None, error seen).  Rows the
    library leaves untouched are 0 in the returned q."""
    pool = pool.copy()
    q_out = None if q_bits is None else np.zeros_like(q_bits)
    T, (S, M), pages = k_bits.shape[0], tables.shape, pool.shape[0]
    err = False
    for s in range(len(lens)):
        lo, hi, n = int(cu[s]), int(cu[s + 1]), int(lens[s])
        if hi <= lo:
            continue
        if hi > T or n < hi - lo or n > M * PAGE_TOKENS or (cos is not None and n > cos.shape[0]):
            err = True
            continue
        for t in range(lo, hi):
            pos = n - (hi - t)
            page = int(tables[s, pos // PAGE_TOKENS])
            if not 0 <= page < pages:
                err = True
                continue
            k = k_bits[t]
            if cos is not None:
                k = rope.rotate_bf16(k, cos[pos], sin[pos])
                if q_bits is not None:
                    q_out[t] = rope.rotate_bf16(q_bits[t], cos[pos], sin[pos])
            for kv, rows in ((0, k), (1, v_bits[t])):
                codes, scale, low = quantise(rows)
                for g in range(NUM_KV_HEADS):
                    write_row(pool[page, g], kv, pos % PAGE_TOKENS, codes[g], scale[g], low[g])
    return pool, q_out, err


def attend(q_bits, pool, tables, lens, scale):
    """FP64 attention and the sizes its error bounds are made of, per output: (out,
    sum of p (15 scale + |lo|) of V over sum of p; per head: the largest |scale|
    sum |q| (15 scale + |lo|) of K, the largest 15 scale + |lo| of V)."""
    S = len(lens)
    out = np.zeros((S, NUM_Q_HEADS, HEAD_DIM))
    size, reach, most = (np.zeros((S, NUM_Q_HEADS, 1)) for _ in range(3))
    q = bf16.to_f64(q_bits)
    for s in range(S):
        n = int(lens[s])
        if n <= 0 or n > tables.shape[1] * PAGE_TOKENS:
            continue
        ids = tables[s, :-(-n // PAGE_TOKENS)]
        if (ids < 0).any() or (ids >= pool.shape[0]).any():
            continue
        c, sc, lo = codes_of(pool[ids])
        kv = (lo[..., None] + c * sc[..., None]).transpose(2, 1, 0, 3, 4).reshape(2, NUM_KV_HEADS, -1, HEAD_DIM)[:, :, :n]
        span = (15 * sc + np.abs(lo)).transpose(2, 1, 0, 3).reshape(2, NUM_KV_HEADS, -1)[:, :, :n]
        for h in range(NUM_Q_HEADS):
            k, v = kv[0, h // GROUP], kv[1, h // GROUP]
            x = scale * (k @ q[s, h])
            p = np.exp(x - x.max())
            out[s, h] = p @ v / p.sum()
            size[s, h] = p @ span[1, h // GROUP] / p.sum()
            reach[s, h] = abs(scale) * np.abs(q[s, h]).sum() * span[0, h // GROUP].max()
            most[s, h] = span[1, h // GROUP].max()
    return out, size, reach, most
