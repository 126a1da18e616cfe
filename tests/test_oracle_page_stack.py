"""The oracle of block tables that grow on the GPU against the admission oracle's
scheduler: the same pages in the same order, and the same stack after releases."""
import numpy as np
import pytest

from oracle import admission as A, page_stack as PS


@pytest.mark.parametrize("layers,seed", [(1, 0), (3, 1), (16, 2)])
def test_pages_are_those_of_the_scheduler(layers, seed):
    g = np.random.default_rng(seed)
    rows, width, pages = 5, 6, layers * 30
    sched = A.Scheduler(pages, layers, width, rows)
    for _ in range(rows):
        sched.submit(60, 30)
    assert len(sched.admit()) == rows
    tables = np.full((layers, rows, width), -1, np.int32)
    lens, stack, count = np.zeros(rows, np.int32), np.arange(pages - 1, -1, -1, dtype=np.int32), pages
    for step in range(4):
        new = g.integers(0, 20, rows)
        tables, lens, count, cu, pos, seq, slots, err = PS.grow(lens, new, tables, stack, count)
        assert err == 0 and cu[-1] == new.sum() == len(pos)
        for s in range(rows):
            assert sched.grow(s, int(lens[s])) == A.Scheduler.OK
            for layer in range(layers):
                want = sched.req[s]["pages"][layer]
                assert list(tables[layer, s, :PS.blocks(int(lens[s]))]) == list(want)
        assert count == len(sched.free) and list(stack[:count]) == sched.free
        for t in range(len(pos)):
            assert pos[t] == lens[seq[t]] - new[seq[t]] + t - cu[seq[t]]
            assert np.array_equal(slots[:, t], tables[:, seq[t], pos[t] // 16] * 16 + pos[t] % 16)
    done = np.array([1, 0, 1, 0, 0])
    stack, lens, count, err = PS.release(lens, done, tables, stack, count)
    for s in (0, 2):
        sched.finish(s)
    assert err == 0 and list(stack[:count]) == sched.free and lens[0] == lens[2] == 0


def test_refusals_change_nothing():
    tables, stack = np.full((2, 2, 2), -1, np.int32), np.arange(6, dtype=np.int32)
    for new, count, T, err in (([33, 0], 6, None, PS.BAD), ([-1, 0], 6, None, PS.BAD), ([3, 2], 6, 4, PS.BAD),
                               ([1, 1], 7, None, PS.BAD), ([32, 17], 6, None, PS.EXHAUSTED)):
        got = PS.grow([0, 0], new, tables, stack, count, T)
        assert got[-1] == err and np.array_equal(got[0], tables) and got[2] == count and not got[3].any()
        assert (got[4] == -1).all() and (got[6] == -1).all()
    tables[:, 0, 0] = [4, 9]
    assert PS.release([5, 0], [1, 0], tables, stack, 0)[-1] == PS.BAD
    tables[:, 0, 0] = [4, 5]
    assert PS.release([5, 0], [1, 0], tables, stack, 5)[-1] == PS.BAD
    assert PS.release([5, 0], [1, 0], tables, stack, 4)[2:] == (6, 0)
