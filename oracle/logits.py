"""Penalties, biases and masks on logits, and the next token (test
infrastructure only), token by token in fp32 as the library defines them:

    in the history:          x = x / repetition if x > 0 else x * repetition
    n > 0 times generated:   x = x - frequency * n, then x = x - presence
    with a bias entry:       x = x + bias   (the last entry of an id)
    masked out:              x = -inf
and the first index of the largest non-NaN x that is not masked out, or -1.
Every operation is rounded to fp32.
"""
from __future__ import annotations

import numpy as np

f32 = np.float32


def process(logits, history=None, history_lens=None, prompt_lens=None, repetition=None, presence=None,
            frequency=None, bias_ids=None, bias_values=None, mask=None):
    """logits float32 [rows][vocab] (already widened); returns (logits, ids)."""
    out = np.array(logits, dtype=f32)
    rows, vocab = out.shape
    ids = np.full(rows, -1, np.int32)
    with np.errstate(all="ignore"):
        for r in range(rows):
            x = out[r]
            if history is not None:
                n = min(max(int(history_lens[r]), 0), history.shape[1])
                start = 0 if prompt_lens is None else int(prompt_lens[r])
                count, seen = {}, set()
                for k in range(n):
                    i = int(history[r, k])
                    if 0 <= i < vocab:
                        seen.add(i)
                        if k >= start:
                            count[i] = count.get(i, 0) + 1
                rep = f32(1) if repetition is None else f32(repetition[r])
                pres = f32(0) if presence is None else f32(presence[r])
                freq = f32(0) if frequency is None else f32(frequency[r])
                for i in seen:
                    x[i] = f32(x[i] / rep) if x[i] > 0 else f32(x[i] * rep)
                    if i in count:
                        x[i] = f32(x[i] - f32(freq * f32(count[i])))
                        x[i] = f32(x[i] - pres)
            if bias_ids is not None:
                last = {int(i): f32(v) for i, v in zip(bias_ids[r], bias_values[r]) if 0 <= i < vocab}
                for i, v in last.items():
                    x[i] = f32(x[i] + v)
            allowed = np.ones(vocab, bool)
            if mask is not None:
                words = np.asarray(mask[r]).view(np.uint32)
                i = np.arange(vocab)
                allowed = ((words[i >> 5] >> (i & 31).astype(np.uint32)) & 1).astype(bool)
                x[~allowed] = -np.inf
            can = np.flatnonzero(allowed & ~np.isnan(x))
            if len(can):
                ids[r] = can[np.argmax(x[can])]
    return out, ids
