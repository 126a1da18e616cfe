"""Attention over 4-bit pages (paged_gqa_decode_int4) against the FP64 oracle.

With A = sum p (15 scale + |lo|) / sum p over V's rows and R = |scale| sum |q| (15
scale + |lo|) over K's largest row, an output may be off by
  its own rounding, 2^-8 of the value;
  a score: 64 products summed by the tensor core, at most 2^-23 a step, 16 + 2 steps
  for the sum of q, and a dozen operations around them, 2^-24 each: less than
  2^-16 R, in numerator and denominator;
  an exponential 2^-22, the products with scale and lift and the two fp16 columns
  2^-22, the logarithm of a weight 2^-22 in each of two merges: 2^-20 A, in both;
  the sums: a page's product 16 steps of 2^-23, one addition per page, 8 warps, up to 8
  CTAs or the parts of a merge: (n / 16 + 64) 2^-23 A;
  the least step of fp16, 2^-24, half of it for either column, on weights whose largest
  is at least 2^13: n 2^-37 of the largest row.
"""
import numpy as np
import pytest
import torch

from oracle import bf16 as OB, int4_kv as O4
from tests._util import bits, to_dev_bf16, to_dev_i32
from tests.test_gpu_bs8 import rows, tables_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib(cuda_device):
    from paged_kv_gqa_append_gb300 import build
    build.build()
    import paged_kv_gqa_append_gb300 as m
    return m


def random_pages(seed, pages):
    """Any codes under scales and minima as rows of a model have them."""
    g = np.random.default_rng(seed)
    pool = g.integers(0, 256, (pages, 8, O4.BLOCK_BYTES)).astype(np.uint8)
    scale = np.exp(g.normal(-1.2, 0.4, (pages, 8, 32))).astype(np.float32)
    low = (-scale * g.uniform(5, 9, scale.shape)).astype(np.float32)
    put_rows(pool, scale, low)
    return pool


def put_rows(pool, scale, low):
    """scale, low [pages][8][32], in the order of the block's words."""
    pair = np.stack([OB.from_f32_rne(scale), OB.from_f32_rne(low)], -1)
    pool[:, :, 1024:] = np.ascontiguousarray(pair).view(np.uint8).reshape(*pool.shape[:2], 128)


def rows_of(pool, page, kv):
    """The words (scale, minimum) of a page's K or V rows, for changing them: [8][16][2] uint16."""
    at = O4.SCALE_AT[kv][:, None] + np.arange(4)
    return pool[page][:, at].copy().view(np.uint16)


def set_rows(pool, page, kv, words):
    at = O4.SCALE_AT[kv][:, None] + np.arange(4)
    pool[page][:, at] = np.ascontiguousarray(words, dtype=np.uint16).view(np.uint8)


def decode(lib, dev, q, pool, bt, lens, scale=0.125, **kw):
    qd = to_dev_bf16(q, dev)
    out, err = torch.full_like(qd, 5.0), torch.zeros(1, dtype=torch.int32, device=dev)
    pool = pool if isinstance(pool, torch.Tensor) else torch.from_numpy(pool).to(dev)
    lib.paged_gqa_decode_int4(qd, pool, to_dev_i32(bt, dev), to_dev_i32(lens, dev), out, scale, d_err=err, **kw)
    return out, lib.pkv_read_device_error(err)


def close(out, ref, size, reach, most, lens, what=""):
    got = OB.to_f64(bits(out))
    n = np.asarray(lens, np.float64).clip(0)[:, None, None]
    tol = 2.0 ** -8 * np.abs(ref) + (2 * (2.0 ** -16 * reach + 2.0 ** -20) + (n / 16 + 64) * 2.0 ** -23) * size
    tol += n * 2.0 ** -37 * most
    assert np.isfinite(got).all(), what
    over = np.abs(got - ref) - tol * (1 + 2.0 ** -8) - 1e-38
    assert (over <= 0).all(), f"{what}: {over.max():.3e} over at {np.unravel_index(over.argmax(), over.shape)}"


def check(lib, dev, q, pool, bt, lens, scale=0.125, **kw):
    out, code = decode(lib, dev, q, pool, bt, lens, scale, **kw)
    assert code == 0
    close(out, *O4.attend(q, pool, bt, lens, scale), lens)
    return out


@pytest.mark.parametrize("lens", [[1], [15], [16], [17], [31], [32], [33], [37], [49], [64], [65], [129], [2048], [2047],
                                  [0], [0, 0, 5, 0], [1] * 40, [2048, 1, 0, 700, 17, 1500, 2047, 129],
                                  [33, 600, 0, 16, 16, 16, 999], list(range(70)), [9000], [5000, 17, 0, 4999]])
def test_lengths(lib, cuda_device, lens):
    pages = sum(-(-n // 16) for n in lens) + 2
    pool = random_pages(30, pages)
    bt = tables_for(31, lens, pages)
    pool[np.setdiff1d(np.arange(pages), bt)] = 0xFF          # pages of nobody: NaN scales
    for s, n in enumerate(lens):                             # rows behind the end hold anything, NaN and infinities among it
        if n % 16:
            for kv in range(2):
                w = rows_of(pool, bt[s, n // 16], kv)
                w[:, n % 16:] = [0x7FC0, 0x7F80] if s % 2 else [0x7F7F, 0xFFC0]
                set_rows(pool, bt[s, n // 16], kv, w)
    q = rows(32, len(lens), 32, 64)
    # whole sequences, and (by a bound that they would be too long for) shares
    for bound in (max(lens), 1 << 20):
        out = check(lib, cuda_device, q, pool, bt, lens, max_seq_len=bound)
        again, _ = decode(lib, cuda_device, q, pool, bt, lens, max_seq_len=bound)
        assert torch.equal(out.view(torch.int16), again.view(torch.int16))
        for s, n in enumerate(lens):
            if n == 0:
                assert (out[s] == 0).all()


def test_long_sequence_and_wrong_bounds(lib, cuda_device):
    lens = [20011, 3]
    pool = random_pages(33, 1300)
    bt = tables_for(34, lens, 1300, 1400)
    q = rows(35, 2, 32, 64, scale=0.5)
    check(lib, cuda_device, q, pool, bt, lens)
    check(lib, cuda_device, q, pool, bt, lens, max_seq_len=16)         # a bound far too small
    check(lib, cuda_device, q, pool, bt, lens, max_blocks=1251, max_seq_len=0)


@pytest.mark.parametrize("bound", [160, 1 << 20])
@pytest.mark.parametrize("what", ["sharp", "tiny q", "huge q", "zero q", "no scale", "negative scale", "outlier V rows",
                                  "outlier K rows", "flat rows", "zero pages", "large V", "largest V", "small V",
                                  "subnormal minima", "large K", "ascending scores", "positive rows", "heads far apart",
                                  "ascending V, falling scores", "cancelling"])
def test_values(lib, cuda_device, what, bound):
    lens = [150, 47]
    pool = random_pages(36, 16)
    bt = tables_for(37, lens, 16)
    q, scale = rows(38, 2, 32, 64), 0.125
    every = range(16)

    def times(kv, page, by, at=slice(None)):
        w = rows_of(pool, page, kv)
        w[:, at] = OB.from_f32_rne((OB.to_f64(w[:, at]) * by).astype(np.float32))
        set_rows(pool, page, kv, w)
    if what == "sharp":
        q = rows(38, 2, 32, 64, scale=20.0)
    elif what == "tiny q":
        q = rows(38, 2, 32, 64, scale=1e-36)
    elif what == "huge q":
        q, scale = rows(38, 2, 32, 64, scale=1e30), 1e-31
    elif what == "zero q":
        q = q & 0x8000
    elif what == "no scale":
        scale = 0.0
    elif what == "negative scale":
        scale = -0.2
    elif what == "outlier V rows":
        times(1, bt[0, 3], 2.0 ** 30, slice(5, 7))
        times(1, bt[1, 0], 2.0 ** 20, 0)                     # the first token's
        times(1, bt[1, 2], 2.0 ** -60, slice(0, 9))
    elif what == "outlier K rows":
        times(0, bt[0, 5], 30, 3)
        times(0, bt[1, 1], 200, 15)
    elif what == "flat rows":
        for p in every:
            w = rows_of(pool, p, p % 2)
            w[:, ::2, 0] = 0
            set_rows(pool, p, p % 2, w)
    elif what == "zero pages":
        pool[:] = 0
    elif what == "large V":
        for p in every:
            times(1, p, 1e30)
    elif what == "largest V":                                # rows from -3.4e38 to 3.4e38
        for p in every:
            w = rows_of(pool, p, 1)
            w[..., 1] = 0xFF7F
            w[..., 0] = OB.from_f32_rne(np.float32(3.389e38 / 15 * 2))
            set_rows(pool, p, 1, w)
    elif what == "small V":
        for p in every:
            times(1, p, 1e-30)
            times(0, p, 1e-25)
    elif what == "subnormal minima":
        for p in every:
            w = rows_of(pool, p, 1)
            w[..., 0], w[..., 1] = 0x0080, 0x8003            # 2^-126, -3 2^-133
            set_rows(pool, p, 1, w)
    elif what == "large K":
        for p in every:
            times(0, p, 2.0 ** 110)
        q, scale = rows(38, 2, 32, 64, scale=2.0 ** -110), 0.125
    elif what == "ascending scores":                         # the reference moves at every page
        q = np.abs(OB.to_f64(q))
        q = OB.from_f32_rne(q.astype(np.float32))
        for s in range(2):
            for i, p in enumerate(bt[s][bt[s] >= 0]):
                w = rows_of(pool, p, 0)
                w[..., 1] = OB.from_f32_rne(((i * 16 + np.arange(16)) * 0.5 - 40).astype(np.float32))
                set_rows(pool, p, 0, w)
    elif what == "positive rows":
        for p in every:
            for kv in range(2):
                times(kv, p, -1)
    elif what == "heads far apart":
        q = OB.from_f32_rne((OB.to_f64(q) * 2.0 ** (-22.0 * (np.arange(32) % 4))[:, None]).astype(np.float32))
    elif what == "ascending V, falling scores":
        q = OB.from_f32_rne(np.abs(OB.to_f64(q)).astype(np.float32))
        for s in range(2):
            for i, p in enumerate(bt[s][bt[s] >= 0]):
                k, v = rows_of(pool, p, 0), rows_of(pool, p, 1)
                at = i * 16 + np.arange(16)
                k[..., 1] = OB.from_f32_rne((-0.3 * at).astype(np.float32))
                v[..., 0] = OB.from_f32_rne(np.exp2(0.6 * at).astype(np.float32))
                v[..., 1] = 0
                set_rows(pool, p, 0, k)
                set_rows(pool, p, 1, v)
    elif what == "cancelling":                               # minima that codes of 8 make up for
        for p in every:
            pool[p, :, 512:1024] = 0x88
            w = rows_of(pool, p, 1)
            w[..., 1] = OB.from_f32_rne((-8 * OB.to_f64(w[..., 0])).astype(np.float32))
            set_rows(pool, p, 1, w)
    check(lib, cuda_device, q, pool, bt, lens, scale, max_seq_len=bound)


@pytest.mark.parametrize("bound", [160, 1 << 20])
def test_one_token_gives_its_values(lib, cuda_device, bound):
    """A softmax over one token is 1: the output is bf16(lo + code scale) but for the last place."""
    pool, q = random_pages(70, 3), rows(71, 3, 32, 64)
    bt = np.array([[0], [1], [2]], np.int32)
    out, _ = decode(lib, cuda_device, q, pool, bt, [1, 1, 1], max_seq_len=bound)
    want = O4.values(pool)[:, 1, :, 0].repeat(4, 1)
    err = np.abs(OB.to_f64(bits(out)) - want)
    c, s, lo = O4.codes_of(pool)
    size = (15 * s + np.abs(lo))[:, :, 1, 0].repeat(4, 1)[..., None]
    assert (err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * size).all()


@pytest.mark.parametrize("bound", [160, 1 << 20])
def test_infinite_and_nan_queries_stay_in_their_head(lib, cuda_device, bound):
    lens = [150, 20]
    pool = random_pages(55, 14)
    bt = tables_for(56, lens, 14)
    q = rows(57, 2, 32, 64, scale=1e-3)
    ref = O4.attend(q, pool, bt, lens, 0.125)
    bad = q.copy()
    bad[0, 5, 3], bad[1, 30, 63] = 0x7F80, 0x7FC0          # inf, NaN
    out, code = decode(lib, cuda_device, bad, pool, bt, lens, max_seq_len=bound)
    assert code == 0
    keep = np.ones((2, 32), bool)
    keep[0, 5] = keep[1, 30] = False
    assert torch.isnan(out[1, 30].float()).all() and torch.isnan(out[0, 5].float()).all()
    out[0, 5], out[1, 30] = 0, 0
    close(out, *[r * keep[..., None] for r in ref], lens)


@pytest.mark.parametrize("kv", [0, 1])
@pytest.mark.parametrize("bound", [160, 1 << 20])
def test_rows_that_are_not_finite_show_in_their_group(lib, cuda_device, kv, bound):
    lens = [150, 20]
    pool = random_pages(58, 14)
    bt = tables_for(59, lens, 14)
    q = rows(60, 2, 32, 64)
    ref = O4.attend(q, pool, bt, lens, 0.125)
    w = rows_of(pool, bt[0, 4], kv)
    w[3, 11] = 0x7FC0
    set_rows(pool, bt[0, 4], kv, w)
    out, _ = decode(lib, cuda_device, q, pool, bt, lens, max_seq_len=bound)
    assert torch.isnan(out[0, 12:16].float()).all()
    out[0, 12:16] = 0
    keep = np.ones((2, 32, 1))
    keep[0, 12:16] = 0
    close(out, *[r * keep for r in ref], lens)


@pytest.mark.parametrize("bound", [512, 0])
def test_bad_sequences_alone_are_refused(lib, cuda_device, bound):
    lens = [40, 300, -1, 7000, 2 ** 31 - 1, 500, 33, 20]
    pool = random_pages(39, 60)
    q = rows(40, len(lens), 32, 64)
    bt = np.full((len(lens), 32), -1, np.int32)
    perm = np.random.default_rng(41).permutation(60).astype(np.int32)
    bt[0, :3], bt[1, :19], bt[5, :32], bt[7, :2] = perm[:3], perm[3:22], perm[22:54], perm[54:56]
    bt[5, 17] = 60                                     # outside the pool, in the middle of a split sequence
    bt[6, :2] = perm[56:58]                            # and its third page missing
    for more in (dict(max_seq_len=bound), dict(max_seq_len=1 << 20)):
        out, code = decode(lib, cuda_device, q, pool, bt, lens, **more)
        assert code == lib.ERR_DEVICE_INDEX
        good = [0, 1, 7]
        assert (out[[2, 3, 4, 5, 6]] == 0).all()
        close(out[good], *O4.attend(q[good], pool, bt[good], np.array(lens)[good], 0.125), np.array(lens)[good])


@pytest.mark.parametrize("S", [31, 128, 129, 300])
def test_many_sequences_long_short_empty_and_bad(lib, cuda_device, S):
    g = np.random.default_rng(60 + S)
    lens = g.integers(0, 500, S)
    lens[g.permutation(S)[:S // 3]] = g.integers(0, 18, S // 3)
    lens[[5, S - 2]] = 9001, 6007
    lens[[0, S - 1]] = 0, 700
    pages = int(sum(-(-n // 16) for n in lens)) + 1
    pool = random_pages(61, pages)
    bt = tables_for(62, lens, pages)
    q = rows(63, S, 32, 64)
    for bound in (0, 100):
        check(lib, cuda_device, q, pool, bt, lens, max_seq_len=bound)
    bad = [5, 17, 18, 30, S - 1]
    lens[[17, 18, 30]] = -3, bt.shape[1] * 16 + 1, 480
    bt[5, 300], bt[S - 1, 43], bt[30, :30] = pages, -1, -1
    good = np.setdiff1d(np.arange(S), bad)
    want = O4.attend(q[good], pool, bt[good], lens[good], 0.125)
    for bound in (0, 100):
        out, code = decode(lib, cuda_device, q, pool, bt, lens, max_seq_len=bound)
        assert code == lib.ERR_DEVICE_INDEX
        assert (out[bad] == 0).all()
        close(out[good], *want, lens[good])


def test_largest_batch_and_page_order(lib, cuda_device):
    S = 4096
    lens = np.random.default_rng(42).integers(0, 20, S).astype(np.int32)
    pages = int(sum(-(-n // 16) for n in lens))
    pool = random_pages(43, pages)
    bt = tables_for(44, lens, pages)
    q = rows(45, S, 32, 64)
    perm = np.random.default_rng(46).permutation(pages)      # the same pages elsewhere
    moved = np.empty_like(pool)
    moved[perm] = pool
    bt2 = np.where(bt >= 0, perm[bt.clip(0)], -1).astype(np.int32)
    for bound in (0, 1 << 20):
        out = check(lib, cuda_device, q, pool, bt, lens, max_seq_len=bound)
        out2, _ = decode(lib, cuda_device, q, moved, bt2, lens, max_seq_len=bound)
        assert torch.equal(out.view(torch.int16), out2.view(torch.int16))
    with pytest.raises(lib.PkvError):
        decode(lib, cuda_device, rows(45, S + 1, 32, 64), pool, np.zeros((S + 1, 2), np.int32),
               np.zeros(S + 1, np.int32), workspace=torch.empty(1 << 27, dtype=torch.uint8, device=cuda_device))


def test_shares_longer_than_the_list_of_ids(lib, cuda_device):
    """One CTA's share of more pages than it holds ids of (1024): a table of one page repeated."""
    dev, n = cuda_device, 1 << 20
    pool = random_pages(48, 5)
    S = 8
    bt = np.random.default_rng(49).integers(0, 5, (S, n // 16)).astype(np.int32)
    q = rows(50, S, 32, 64)
    lens = [n, n - 5, n - 16, 17, n, n, 3, n]
    out, code = decode(lib, dev, q, pool, bt, lens)
    assert code == 0
    for s in (1, 3, 6):
        close(out[s:s + 1], *O4.attend(q[s:s + 1], pool, bt[s:s + 1], lens[s:s + 1], 0.125), lens[s:s + 1])


def test_a_cta_for_each_of_many_sequences(lib, cuda_device):
    """By the bound, every sequence is one CTA's: ragged, longer than the bound says (one beyond the
    list of ids), empty, refused."""
    g = np.random.default_rng(72)
    S = 160
    lens = g.integers(0, 300, S)
    lens[[3, 50, S - 1]] = 17000, 0, 700
    pages = int(sum(-(-n // 16) for n in lens)) + 1
    pool = random_pages(73, pages)
    bt = tables_for(74, lens, pages)
    q = rows(75, S, 32, 64)
    check(lib, cuda_device, q, pool, bt, lens, max_seq_len=300)
    bad = [3, 7, 9]
    lens[[7, 9]] = -2, 2 ** 31 - 1
    bt[3, 1030] = pages
    out, code = decode(lib, cuda_device, q, pool, bt, lens, max_seq_len=300)
    assert code == lib.ERR_DEVICE_INDEX and (out[bad] == 0).all() and (out[50] == 0).all()
    good = np.setdiff1d(np.arange(S), bad)
    close(out[good], *O4.attend(q[good], pool, bt[good], lens[good], 0.125), lens[good])


def test_pages_behind_4_gib(lib, cuda_device):
    dev, pages, n = cuda_device, 470000, 100
    pool = torch.empty((pages, 8, O4.BLOCK_BYTES), dtype=torch.uint8, device=dev)
    small = random_pages(58, 7)
    pool[-7:] = torch.from_numpy(small).to(dev)
    q = rows(60, 1, 32, 64)
    bt = np.arange(pages - 7, pages, dtype=np.int32)[None, ::-1].copy()
    for bound in (n, 1 << 20):
        out, code = decode(lib, dev, q, pool, bt, [n], max_seq_len=bound)
        assert code == 0
        close(out, *O4.attend(q, small, np.arange(6, -1, -1, dtype=np.int32)[None], [n], 0.125), [n])


@pytest.mark.parametrize("bound", [0, 1 << 20])
def test_after_a_call_that_leaves_nan_in_shared_memory(lib, cuda_device, bound):
    dev = cuda_device
    big = [2000] * 20
    pool = random_pages(50, 2600)
    bt = tables_for(51, big, 2600)
    lens = [3, 17, 33, 1, 48, 5, 81, 16] * 5
    q = rows(52, len(lens), 32, 64)
    bt2 = tables_for(53, lens, 2600)
    want = O4.attend(q, pool, bt2, lens, 0.125)
    nan = torch.full(pool.shape, 0xFF, dtype=torch.uint8, device=dev)
    for _ in range(3):
        decode(lib, dev, rows(54, 20, 32, 64), nan, bt, big, max_seq_len=bound)
        out, code = decode(lib, dev, q, pool, bt2, lens, max_seq_len=bound)
        assert code == 0
        close(out, *want, lens)


@pytest.mark.parametrize("bound", [1200, 1 << 20])
def test_workspaces_streams_and_graphs(lib, cuda_device, bound):
    """Any content of the workspace; two captured graphs with workspaces of their own
    on two streams at once; replays over other lengths."""
    dev = cuda_device
    lens = [700, 90, 1200, 3]
    pool = random_pages(47, 200)
    bt = tables_for(48, lens, 200, 100)
    q = rows(49, 4, 32, 64)
    want = check(lib, dev, q, pool, bt, lens, max_seq_len=bound)
    d = torch.from_numpy(pool).to(dev)
    n = lib.paged_gqa_decode_int4_workspace_bytes(4)
    graphs = []
    for fill in (0, 255):
        ws = torch.full((n,), fill, dtype=torch.uint8, device=dev)
        a = dict(q=to_dev_bf16(q, dev), out=torch.zeros(4, 32, 64, dtype=torch.bfloat16, device=dev),
                 lens=to_dev_i32(lens, dev), bt=to_dev_i32(bt, dev), ws=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(3):
                lib.paged_gqa_decode_int4(a["q"], d, a["bt"], a["lens"], a["out"], 0.125, workspace=ws, max_seq_len=bound)
        graphs.append((g, a, torch.cuda.Stream(dev)))
    torch.cuda.synchronize(dev)
    for _ in range(5):
        for g, a, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize(dev)
    for g, a, s in graphs:
        assert torch.equal(a["out"].view(torch.int16), want.view(torch.int16))
    short = [16, 90, 0, 3]
    graphs[0][1]["lens"].copy_(to_dev_i32(short, dev))
    graphs[0][0].replay()
    torch.cuda.synchronize(dev)
    close(graphs[0][1]["out"], *O4.attend(q, pool, bt, short, 0.125), short)


def test_refusals(lib, cuda_device):
    dev = cuda_device
    pool = lib.new_int4_pool(4, dev)
    q = torch.zeros(2, 32, 64, dtype=torch.bfloat16, device=dev)
    bt, lens = torch.zeros(2, 3, dtype=torch.int32, device=dev), torch.ones(2, dtype=torch.int32, device=dev)

    def call(**kw):
        a = dict(q=q, kv_pool=pool, block_tables=bt, seq_lens=lens, out=torch.empty_like(q), scale=0.125) | kw
        lib.paged_gqa_decode_int4(**a)
    call()
    for kw, e in ((dict(kv_pool=pool.view(torch.int8)), TypeError), (dict(kv_pool=pool.cpu()), ValueError),
                  (dict(kv_pool=pool[:, :1]), ValueError), (dict(seq_lens=lens[:1]), ValueError),
                  (dict(block_tables=bt[:1]), ValueError), (dict(q=q.float()), TypeError),
                  (dict(scale=float("inf")), lib.PkvError), (dict(max_blocks=4), lib.PkvError),
                  (dict(workspace=torch.empty(64, dtype=torch.uint8, device=dev)), lib.PkvError)):
        with pytest.raises(e):
            call(**kw)
    k = torch.zeros(2, 8, 64, dtype=torch.bfloat16, device=dev)
    cu = torch.arange(3, dtype=torch.int32, device=dev)
    cos = torch.zeros(16, 32, device=dev)
    for kw, e in ((dict(rope_cos=cos), ValueError), (dict(q_in=q, q_out=q), ValueError),
                  (dict(cu_new=cu[:2]), ValueError), (dict(k=k[:1]), ValueError),
                  (dict(rope_cos=cos, rope_sin=cos[:8]), ValueError),
                  (dict(k=k[:, :, :32]), ValueError), (dict(max_blocks=9), lib.PkvError)):
        a = dict(k=k, v=k, cu_new=cu, seq_lens=lens, block_tables=bt, kv_pool=pool) | kw
        with pytest.raises(e):
            lib.kv_append_rope_int4(**a)
    with pytest.raises(ValueError):
        lib.kv_read_int4(pool, bt[0], torch.empty(1, 2, 8, 16, 64, dtype=torch.bfloat16, device=dev))
