"""Block tables that grow and shrink by a stack of free pages (test
infrastructure only), page by page as the admission rules hand them out: the
stack is LIFO, a call goes row by row, in a row layer by layer, in a layer in
order.  Both calls are all or nothing.

Arrays: tables int32 [layers][rows][width]; stack int32 [pages] with `count` free
ids at its front, the last of them taken first.
"""
from __future__ import annotations

import numpy as np

PAGE_TOKENS = 16
OK, BAD, EXHAUSTED = 0, 6, 7


def blocks(n):
    return -(-n // PAGE_TOKENS)


def grow(lens, new, tables, stack, count, T=None):
    """(tables, lens, count, cu, positions, token_seq, slots, error) on copies; T rows
    of positions, token_seq and slots (None: as many as there are new tokens)."""
    tables, (L, S, M) = tables.copy(), tables.shape
    total = int(sum(max(0, int(x)) for x in new))
    T = total if T is None else T
    pos, seq, slots = np.full(T, -1, np.int32), np.full(T, -1, np.int32), np.full((L, T), -1, np.int32)
    keep = tables, np.array(lens, np.int32), count, np.zeros(S + 1, np.int32), pos, seq, slots
    if any(n < 0 or m < 0 or n + m > M * PAGE_TOKENS for n, m in zip(lens, new)) or total > T or not 0 <= count <= len(stack):
        return (*keep, BAD)
    if sum(L * (blocks(n + m) - blocks(n)) for n, m in zip(lens, new)) > count:
        return (*keep, EXHAUSTED)
    free, cu, t, err = list(stack[:count]), [0], 0, OK
    for s in range(S):
        n, m = int(lens[s]), int(new[s])
        for layer in range(L):
            for b in range(blocks(n), blocks(n + m)):
                tables[layer, s, b] = free.pop()
                if not 0 <= tables[layer, s, b] < len(stack):
                    err = BAD
        for p in range(n, n + m):
            pos[t], seq[t] = p, s
            for layer in range(L):
                page = int(tables[layer, s, p // PAGE_TOKENS])
                if 0 <= page < len(stack):
                    slots[layer, t] = page * PAGE_TOKENS + p % PAGE_TOKENS
                else:
                    err = BAD
            t += 1
        cu.append(t)
    return tables, np.array([n + m for n, m in zip(lens, new)], np.int32), len(free), np.array(cu, np.int32), pos, seq, slots, err


def release(lens, done, tables, stack, count):
    """(stack, lens, count, error) on copies."""
    L, S, M = tables.shape
    lens, back = np.array(lens, np.int32), []
    ok = 0 <= count <= len(stack)
    for s in range(S):
        if not done[s]:
            continue
        ok = ok and 0 <= lens[s] <= M * PAGE_TOKENS
        for layer in range(L):
            for b in range(blocks(int(lens[s])) if ok else 0):
                back.append(int(tables[layer, s, b]))
    if not ok or count + len(back) > len(stack) or any(not 0 <= p < len(stack) for p in back):
        return stack.copy(), lens, count, BAD
    stack = stack.copy()
    stack[count:count + len(back)] = back
    return stack, np.where(np.asarray(done, bool), 0, lens).astype(np.int32), count + len(back), OK
