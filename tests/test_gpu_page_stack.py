"""Block tables that grow and shrink on the GPU against the oracle: every integer
equal, for one row to thousands, one layer to many, strides, padding, refusals,
in place, captured and replayed, and against the host scheduler."""
import numpy as np
import pytest
import torch

from oracle import page_stack as PS
from tests._util import to_dev_i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib(cuda_device):
    from paged_kv_gqa_append_gb300 import build
    build.build()
    import paged_kv_gqa_append_gb300 as m
    return m


def start(seed, layers, lens, width, spare=7):
    """Tables [layers][rows][width] of shuffled pages for these lengths, -1 behind them, and the stack of the rest."""
    g = np.random.default_rng(seed)
    need = [PS.blocks(int(n)) for n in lens]
    pages = layers * sum(need) + spare
    ids = g.permutation(pages).astype(np.int32)
    tables = np.full((layers, len(lens), width), -1, np.int32)
    at = 0
    for layer in range(layers):
        for s, n in enumerate(need):
            tables[layer, s, :n] = ids[at:at + n]
            at += n
    stack = np.concatenate([ids[at:], np.full(at, -7, np.int32)])
    return tables, stack, pages - at


class State:
    """A call's buffers on the device; out of place if `apart`."""

    def __init__(self, dev, lens, tables, stack, count, T, apart):
        self.lens, self.count = to_dev_i32(lens, dev), to_dev_i32([count], dev)
        self.tables, self.stack = to_dev_i32(tables, dev), to_dev_i32(stack, dev)
        self.lens_to = torch.full_like(self.lens, 77) if apart else self.lens
        self.count_to = torch.full_like(self.count, 77) if apart else self.count
        self.pos, self.seq = (torch.full((T,), 55, dtype=torch.int32, device=dev) for _ in range(2))
        self.slots = torch.full((tables.shape[0], T), 55, dtype=torch.int32, device=dev)
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)

    def grow(self, lib, new, **kw):
        return lib.grow_block_tables(self.lens, new, self.tables, self.stack, self.count, self.lens_to, self.count_to,
                                     positions=self.pos, token_seq=self.seq, slots=self.slots, d_err=self.err, **kw)

    def release(self, lib, done):
        lib.release_pages(self.lens, done, self.tables, self.stack, self.count, self.lens_to, self.count_to, d_err=self.err)


def equal(got, want):
    assert np.array_equal(got.cpu().numpy(), np.asarray(want))


CASES = [  # layers, rows, held up to, new up to, spare rows of the outputs
    (1, 1, 0, 1, 0), (1, 1, 15, 1, 3), (1, 1, 16, 1, 0), (2, 1, 0, 1000, 5), (16, 32, 2047, 1, 0), (16, 32, 40, 0, 9),
    (3, 33, 100, 37, 1), (28, 64, 0, 300, 0), (7, 1000, 50, 3, 11), (1, 4096, 20, 40, 0), (2, 4096, 33, 1, 2), (16, 257, 64, 33, 40)]


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("layers,rows,held,most,pad", CASES)
def test_grow_and_release(lib, cuda_device, layers, rows, held, most, pad, apart):
    g = np.random.default_rng([layers, rows, held, most])
    lens, new = g.integers(0, held + 1, rows), g.integers(0, most + 1, rows)
    new[g.integers(rows)] = most
    width = PS.blocks(int((lens + new).max())) + 1
    extra = layers * int(sum(PS.blocks(int(n + m)) - PS.blocks(int(n)) for n, m in zip(lens, new)))
    tables, stack, count = start(rows, layers, lens, width, extra + 3)
    T = int(new.sum()) + pad
    st = State(cuda_device, lens, tables, stack, count, T, apart)
    for _ in range(2 if apart else 1):  # out of place: the same again
        cu = st.grow(lib, to_dev_i32(new, cuda_device))
    want = PS.grow(lens, new, tables, stack, count, T)
    assert want[-1] == 0
    for got, w in zip((st.tables, st.lens_to, st.count_to, cu, st.pos, st.seq, st.slots), want):
        equal(got.view(-1), np.ravel(w))
    equal(st.err, [0])
    if apart:
        equal(st.lens, lens)
        equal(st.count, [count])
    # about half of them finished
    done = g.random(rows) < 0.5
    done[0] = True
    st2 = State(cuda_device, want[1], want[0], stack, want[2], 0, apart)
    st2.release(lib, torch.from_numpy(done).to(cuda_device))
    back = PS.release(want[1], done, want[0], stack, want[2])
    assert back[-1] == 0
    equal(st2.count_to, [back[2]])
    equal(st2.stack[:back[2]], back[0][:back[2]])
    equal(st2.stack[back[2]:], stack[back[2]:])  # above the stack nothing is written
    equal(st2.lens_to, back[1])
    equal(st2.tables, want[0])
    equal(st2.err, [0])


@pytest.mark.parametrize("rows", [3, 3000])
def test_grow_refusals_are_all_or_nothing(lib, cuda_device, rows):
    lens = np.full(rows, 20)
    tables, stack, count = start(5, 2, lens, 3, 2 * rows)
    for what, err in (("room", 6), ("negative", 6), ("length", 6), ("T", 6), ("count", 6), ("below", 6), ("pages", 7)):
        new, held, free, T = np.full(rows, 13), lens.copy(), count, 13 * rows
        if what == "room":
            new[-1] = 29
            T += 29
        elif what == "negative":
            new[1] = -1
        elif what == "length":
            held[rows // 2] = -5
        elif what == "T":
            T -= 1
        elif what == "count":
            free = len(stack) + 1
        elif what == "below":
            free = -1
        else:
            free = 2 * rows - 1
        st = State(cuda_device, held, tables, stack, free, T, False)
        cu = st.grow(lib, to_dev_i32(new, cuda_device))
        assert PS.grow(held, new, tables, stack, free, T)[-1] == err
        equal(st.err, [err])
        equal(st.tables, tables)
        equal(st.lens, held)
        equal(st.count, [free])
        assert not cu.any() and (st.pos == -1).all() and (st.seq == -1).all() and (st.slots == -1).all(), what


@pytest.mark.parametrize("rows", [3, 3000])
def test_release_refusals_are_all_or_nothing(lib, cuda_device, rows):
    lens = np.full(rows, 40)
    tables, stack, count = start(6, 2, lens, 3, 4)
    for what in ("id", "minus", "length", "long", "full", "count"):
        held, tb, free = lens.copy(), tables.copy(), count
        if what == "id":
            tb[1, rows - 1, 2] = len(stack)
        elif what == "minus":
            tb[0, 0, 0] = -1
        elif what == "length":
            held[1] = -1
        elif what == "long":
            held[1] = 49
        elif what == "full":
            free = 5
        else:
            free = len(stack) + 1
        done = np.ones(rows, bool)
        st = State(cuda_device, held, tb, stack, free, 0, False)
        st.release(lib, torch.from_numpy(done).to(cuda_device))
        assert PS.release(held, done, tb, stack, free)[-1] == 6
        equal(st.err, [6])
        equal(st.lens, held)
        equal(st.count, [free])
        equal(st.stack[:max(0, min(free, count))], stack[:max(0, min(free, count))])
    # a bad entry of a row that stays is nobody's business
    tb = tables.copy()
    tb[0, 1, 0] = -1
    done = np.zeros(rows, bool)
    done[0] = True
    st = State(cuda_device, lens, tb, stack, count, 0, False)
    st.release(lib, torch.from_numpy(done).to(cuda_device))
    equal(st.err, [0])
    equal(st.count, [count + 6])


def test_ids_on_the_stack_that_cannot_be(lib, cuda_device):
    tables, stack, count = start(7, 2, [5, 0], 2, 6)
    stack[count - 2] = 1000
    st = State(cuda_device, [5, 0], tables, stack, count, 20, False)
    st.grow(lib, to_dev_i32([3, 17], cuda_device))
    want = PS.grow([5, 0], [3, 17], tables, stack, count)
    assert want[-1] == 6
    equal(st.err, [6])
    for got, w in zip((st.tables, st.slots, st.pos), (want[0], want[6], want[4])):
        equal(got, w)


def test_strides_one_token_each_and_missing_outputs(lib, cuda_device):
    """Tables as a slice of a larger allocation, new_tokens None, no positions or slots."""
    dev = cuda_device
    lens = np.array([16, 3, 0, 31])
    tables, stack, count = start(8, 3, lens, 4, 20)
    big = torch.full((5, 6, 9), -3, dtype=torch.int32, device=dev)
    view = big[1:4, :4, 2:6]
    view.copy_(to_dev_i32(tables, dev))
    keep = big.clone()
    L, C, S = to_dev_i32(lens, dev), to_dev_i32([count], dev), to_dev_i32(stack, dev)
    cu = lib.grow_block_tables(L, None, view, S, C)
    want = PS.grow(lens, np.ones(4, int), tables, stack, count)
    equal(view, want[0])
    equal(L, want[1])
    equal(C, [want[2]])
    equal(cu, want[3])
    keep[1:4, :4, 2:6] = view
    assert torch.equal(keep, big)
    one = torch.full((4,), 9, dtype=torch.int32, device=dev)
    lib.grow_block_tables(L, None, view, S, C, positions=one)
    equal(one, want[1])
    lib.release_pages(L, torch.ones(4, dtype=torch.uint8, device=dev), view, S, C)
    equal(L, [0] * 4)
    equal(S[:len(stack)].sort()[0], np.arange(len(stack)))  # every page is back, once
    equal(C, [len(stack)])


def test_no_rows(lib, cuda_device):
    dev = cuda_device
    empty, tables = torch.empty(0, dtype=torch.int32, device=dev), torch.empty((2, 1, 3), dtype=torch.int32, device=dev)
    stack, count = lib.new_free_pages(9, dev)
    equal(lib.grow_block_tables(empty, empty, tables, stack, count), [0])
    lib.release_pages(empty, torch.empty(0, dtype=torch.bool, device=dev), tables, stack, count)
    equal(count, [9])
    equal(stack, np.arange(8, -1, -1))


def test_a_captured_loop_follows_the_host_scheduler(lib, cuda_device):
    """Prompts, then steps of one captured graph with a row that finishes and begins
    anew: tables, lengths and free pages are the Scheduler's."""
    dev, layers, rows, width, pages = cuda_device, 4, 3, 6, 100
    sched = lib.Scheduler(pages, layers, max_blocks=width, max_slots=rows)
    prompts = [30, 1, 17]
    ids = [sched.submit(n, 60)[1] for n in prompts]
    assert len(sched.admit()) == rows
    tables = torch.full((layers, rows, width), -1, dtype=torch.int32, device=dev)
    stack, count = lib.new_free_pages(pages, dev)
    lens, new = torch.zeros(rows, dtype=torch.int32, device=dev), to_dev_i32(prompts, dev)
    done, err = torch.zeros(rows, dtype=torch.bool, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    T = 64
    pos, seq = (torch.empty(T, dtype=torch.int32, device=dev) for _ in range(2))
    slots = torch.empty((layers, T), dtype=torch.int32, device=dev)
    cu = torch.empty(rows + 1, dtype=torch.int32, device=dev)

    def step():
        lib.release_pages(lens, done, tables, stack, count, d_err=err)
        lib.grow_block_tables(lens, new, tables, stack, count, cu_new=cu, positions=pos, token_seq=seq, slots=slots, d_err=err)

    step()
    torch.cuda.synchronize(dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for rid, n in zip(ids, prompts):
        assert sched.grow(rid, n) == 0
    held = list(prompts)
    for t in range(40):
        if t:
            done.zero_()
            new.fill_(1)
            grown = [1] * rows
            if t == 20:  # row 1 finishes, and a request of 25 tokens takes its place
                done[1] = True
                new[1] = 25
                sched.finish(ids[1])
                ids[1] = sched.submit(25, 60)[1]
                assert sched.admit() == [ids[1]]
                held[1], grown[1] = 0, 25
            graph.replay()
            for s in range(rows):
                held[s] += grown[s]
                assert sched.grow(ids[s], held[s]) == 0
        equal(lens, held)
        equal(count, [sched.stats()["free"]])
        for s in range(rows):
            for layer in range(layers):
                n = PS.blocks(held[s])
                row = sched.block_table(ids[s], layer)
                row = row[0] if isinstance(row, tuple) else row
                equal(tables[layer, s, :n], np.asarray(row)[:n])
    equal(err, [0])
