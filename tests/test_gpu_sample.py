"""pkv_sample_logits against the FP64 oracle.  An id has to be the oracle's, or one that
32 bits may give: the sums of w are off by at most 2e-5 of themselves (a hundred additions
of 2^-24 along the longest path, exponentials with arguments below 30 off by 2^-18 where
they count), the race by 2e-5 in the logarithm.  Log-probabilities: 2^-22 of their size (two
roundings and a logarithm), 2e-5 for the sum."""
import numpy as np
import pytest
import torch

from oracle import sampling as S
from tests._util import to_dev_i32

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def lib(cuda_device):
    from paged_kv_gqa_append_gb300 import build
    build.build()
    import paged_kv_gqa_append_gb300 as m
    return m


def f32(x, dev):
    return None if x is None else torch.as_tensor(np.asarray(x, np.float32)).to(dev)


def of_row(a, r, other):
    return other if a is None else float(np.float32(a[r]))


def check(lib, dev, x, noise, T=None, k=None, p=None, floor=None, exact_ids=None):
    """x a torch tensor on the device, noise too; the limits lists of one per row or None."""
    rows = x.shape[0]
    lp = torch.full((rows,), 7.0, device=dev)
    ids = lib.sample_logits(x, noise, temperature=f32(T, dev), top_k=None if k is None else to_dev_i32(k, dev), top_p=f32(p, dev),
                            min_p=f32(floor, dev), logprobs=lp)
    again = lib.sample_logits(x, noise, temperature=f32(T, dev), top_k=None if k is None else to_dev_i32(k, dev),
                              top_p=f32(p, dev), min_p=f32(floor, dev))
    assert torch.equal(ids, again)
    xs, es = x.float().cpu().numpy(), None if noise is None else noise.cpu().numpy()
    got, lps = ids.cpu().numpy(), lp.cpu().numpy()
    for r in range(rows):
        a = dict(T=of_row(T, r, 1.0), k=0 if k is None else int(k[r]), p=of_row(p, r, 1.0), floor=of_row(floor, r, 0.0))
        e = np.ones(x.shape[1]) if es is None else es[r]
        assert S.acceptable(int(got[r]), xs[r], e, **a), (r, got[r], S.sample(xs[r], e, **a), a)
        if got[r] < 0:
            assert np.isnan(lps[r])
            continue
        want = S.limits(xs[r], a["T"] or 1.0)[2][got[r]]
        assert abs(lps[r] - want) <= 2.0 ** -22 * abs(want) + 2e-5, (r, lps[r], want)
    return got


def logits(seed, rows, vocab, dtype, dev, sigma=2.0, near=12):
    g = torch.Generator("cpu").manual_seed(seed)
    x = sigma * torch.randn(rows, vocab, generator=g)
    if near and vocab > 50:
        x[:, torch.randperm(vocab, generator=g)[:near]] += 3 + 3 * torch.rand(rows, near, generator=g)
    return x.to(dtype).to(dev), torch.empty(rows, vocab).exponential_(generator=g).to(dev)


LIMITS = [dict(), dict(k=40), dict(p=0.9), dict(floor=0.05), dict(k=3, p=0.5, floor=0.2), dict(k=2000), dict(k=1), dict(p=0.999),
          dict(p=0.0), dict(floor=1.5), dict(k=10 ** 6, p=1.5, floor=-1.0)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [1, 2, 7, 33, 1000, 4096, 4097, 9999, 32768, 50257, 128256])
def test_sizes_types_and_limits(lib, cuda_device, dtype, vocab):
    rows = 3 if vocab < 20000 else 2
    x, e = logits(vocab, rows, vocab, dtype, cuda_device)
    for i, lim in enumerate(LIMITS):
        T = [0.7, 1.3, 0.0][:rows] if i % 2 else None
        check(lib, cuda_device, x, e, T, **{n: [v] * rows for n, v in lim.items()})


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [0.01, 0.5, 1.0, 5.0, 1e30, 1e-30])
def test_flat_and_sharp_rows(lib, cuda_device, dtype, T):
    """Lists that overflow, bounds that do not hold, everything tied."""
    rows, vocab = 5, 40000
    x, e = logits(3, rows, vocab, dtype, cuda_device, sigma=1.0, near=0)
    x[1] = 0
    x[2] = x[2] * 0.01
    x[3] = -x[3].abs()
    x[4, ::2], x[4, 1::2] = 1.0, -0.0
    for lim in (dict(), dict(p=0.3), dict(p=0.95), dict(k=500), dict(k=3), dict(floor=0.5), dict(k=30000, p=0.99, floor=1e-6)):
        check(lib, cuda_device, x, e, [T] * rows, **{n: [v] * rows for n, v in lim.items()})


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_of_their_own(lib, cuda_device, dtype):
    """Every row with its own limits, some of them off, greedy rows between."""
    g = np.random.default_rng(4)
    rows, vocab = 60, 5003
    x, e = logits(5, rows, vocab, dtype, cuda_device)
    T = np.where(g.random(rows) < 0.2, 0.0, g.uniform(0.3, 2, rows))
    check(lib, cuda_device, x, e, T, k=g.integers(-1, 60, rows), p=g.uniform(0.2, 1.2, rows), floor=g.uniform(-0.1, 0.2, rows))


@pytest.mark.parametrize("vocab", [90, 20000])
def test_values_that_are_not_finite(lib, cuda_device, vocab):
    dev = cuda_device
    x, e = logits(6, 12, vocab, torch.float32, dev)
    x[0], x[1] = -torch.inf, torch.nan
    x[2, 5:] = -torch.inf
    x[3, 7], x[3, 70] = torch.inf, torch.inf
    x[4, ::3] = torch.nan
    x[5, 80] = torch.inf
    e[6, ::2], e[6, 1::2] = 0.0, torch.nan
    e[7] = torch.inf
    e[8] = -1.0
    x[9], x[9, 60] = -3.4e38, 3.4e38
    x[10] = torch.finfo(torch.float32).min
    x[11, ::2] = -torch.inf
    for lim in (dict(), dict(k=4), dict(p=0.7), dict(floor=0.1), dict(k=50, p=0.99, floor=0.001)):
        got = check(lib, dev, x, e, [1.0] * 12, **{n: [v] * 12 for n, v in lim.items()})
        assert got[0] == got[1] == -1 and got[5] == 80 and got[3] in (7, 70) and got[9] == 60
    got = check(lib, dev, x, None, [0.0] * 12)
    assert got[3] == 7 and got[10] == 0
    bad = [-1.0, float("nan"), float("inf"), 1.0, 1.0, 0.0] * 2
    p = [0.9, 0.9, 0.9, float("nan"), 0.9, float("nan")] * 2
    floor = [0.0, 0.0, 0.0, 0.0, float("nan"), 0.0] * 2
    ids = lib.sample_logits(x, e, f32(bad, dev), top_p=f32(p, dev), min_p=f32(floor, dev))
    assert (ids == -1).all()
    assert (lib.sample_logits(x, None, f32([1.0] * 12, dev)) == -1).all()          # rows that draw have no noise


@pytest.mark.parametrize("k,p", [(1, 1.0), (5, 1.0), (0, 0.02), (0, 0.3), (700, 0.9)])
@pytest.mark.parametrize("vocab", [500, 30000])
def test_noise_that_takes_many_rounds(lib, cuda_device, vocab, k, p):
    """Noise that lets the last of any set win: every round takes away one token, until
    the last kept one is bisected for."""
    dev = cuda_device
    x, _ = logits(7, 3, vocab, torch.float32, dev, sigma=0.5, near=0)
    x[1] = torch.round(x[1] * 2) / 2                               # many ties
    x[2] = 0.25
    order = torch.argsort(x, dim=1, descending=True, stable=True)
    rank = torch.empty_like(order).scatter_(1, order, torch.arange(vocab, device=dev).expand(3, -1).contiguous())
    e = torch.exp(80 * (0.5 - (rank + 1) / vocab)).float()
    check(lib, dev, x, e, [1.0] * 3, k=[k] * 3, p=[p] * 3)


def test_strides_and_alignments(lib, cuda_device):
    """Rows that begin anywhere, logits and noise differently."""
    dev, rows, vocab = cuda_device, 9, 5000
    for dtype in TYPES:
        big, noise = logits(8, rows, vocab + 30, dtype, dev)
        for a, b in ((0, 0), (1, 0), (0, 1), (3, 3), (7, 2), (9, 6)):
            x, e = big[:, a:a + vocab + 13], noise[:, b:b + vocab + 13]
            check(lib, dev, x, e, [0.8] * rows, p=[0.9] * rows)
            check(lib, dev, x, e, [0.8] * rows)
            check(lib, dev, x, e, [0.8] * rows, k=[9] * rows)
    tall = big.t().contiguous()[:rows]                             # any shape of rows
    check(lib, dev, tall, noise[:, :rows].contiguous()[:, :rows] if tall.shape[1] == rows else
          torch.empty(tall.shape, device=dev).exponential_(), [1.0] * rows)


def test_large_vocabulary_is_read_again(lib, cuda_device):
    """A part beyond shared memory, and offsets behind 2^31 elements."""
    dev, vocab = cuda_device, 600000
    x, e = logits(9, 2, vocab, torch.float32, dev)
    for lim in (dict(), dict(k=20), dict(p=0.6), dict(p=0.9, floor=1e-4)):
        check(lib, dev, x, e, [0.9] * 2, **{n: [v] * 2 for n, v in lim.items()})
    rows, vocab = 17200, 128256                                    # 2.2 x 10^9 logits
    x = torch.zeros((rows, vocab), dtype=torch.bfloat16, device=dev)
    hot = torch.randint(0, vocab, (rows,), device=dev, generator=torch.Generator(dev).manual_seed(10))
    x.scatter_(1, hot[:, None], 40.0)
    ids = lib.sample_logits(x, None, torch.zeros(rows, device=dev))
    assert torch.equal(ids.long(), hot)


def test_frequencies(lib, cuda_device):
    dev, n = cuda_device, 40000
    x = torch.tensor([1.0, 0.2, 2.0, -1.0, 1.5, 0.2, -3.0, 0.9]).to(dev).expand(n, 8).contiguous()
    e = torch.empty(n, 8, device=dev).exponential_(generator=torch.Generator(dev).manual_seed(11))
    one = torch.ones(n, device=dev)
    for lim, keep in ((dict(), range(8)), (dict(top_k=torch.full((n,), 5, dtype=torch.int32, device=dev)), (0, 1, 2, 4, 7)),
                      (dict(top_p=0.7 * one), (0, 2, 4)), (dict(min_p=0.2 * one), (0, 2, 4, 7))):
        ids = lib.sample_logits(x, e, 0.9 * one, **lim).cpu().numpy()
        w = np.zeros(8)
        w[list(keep)] = np.exp(x[0].cpu().numpy().astype(np.float64)[list(keep)] / 0.9)
        q = w / w.sum()
        assert (np.abs(np.bincount(ids, minlength=8) - n * q) <= 5 * np.sqrt(n * q * (1 - q)) + 1e-9).all(), lim


def test_streams_graphs_and_refusals(lib, cuda_device):
    dev, rows, vocab = cuda_device, 4, 9000
    x, e = logits(12, rows, vocab, torch.float32, dev)
    T, p = f32([0.8] * rows, dev), f32([0.8] * rows, dev)
    want = lib.sample_logits(x, e, T, top_p=p)
    ids, lp = torch.zeros(rows, dtype=torch.int32, device=dev), torch.zeros(rows, device=dev)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.sample_logits(x, e, T, top_p=p, ids=ids, logprobs=lp)
    g.replay()
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    other = lib.sample_logits(x, e, T, top_p=p, stream=side)
    torch.cuda.synchronize(dev)
    assert torch.equal(ids, want) and torch.equal(other, want)
    e.exponential_()
    g.replay()
    assert torch.equal(ids, lib.sample_logits(x, e, T, top_p=p))
    assert lib.sample_logits(x[:0], e[:0]).shape == (0,)
    for kw, err in ((dict(noise=None), ValueError), (dict(noise=e.half()), TypeError), (dict(noise=e[:, :-1]), ValueError),
                    (dict(noise=e.cpu()), ValueError), (dict(logits=x.double()), TypeError), (dict(logits=x.t()), ValueError),
                    (dict(logits=x.cpu()), ValueError), (dict(temperature=T[:1]), ValueError), (dict(top_k=p), TypeError),
                    (dict(top_p=T.double()), TypeError), (dict(ids=ids.long()), TypeError), (dict(logprobs=lp[:2]), ValueError)):
        with pytest.raises(err):
            lib.sample_logits(**(dict(logits=x, noise=e) | kw))


@pytest.mark.parametrize("dtype", TYPES)
def test_many_rows_of_a_large_vocabulary(lib, cuda_device, dtype):
    """More CTAs than two for each SM work in another shape, with limits and without."""
    dev, rows, vocab = cuda_device, 44, 33001
    x, e = logits(13, rows, vocab, dtype, dev)
    x[1::4], x[2::8] = x[1::4] * 0.05, 0.5                         # flat ones, tied ones
    x[3, 5:], x[7] = -torch.inf, torch.nan
    x[11, 7], x[11, 9000] = torch.inf, torch.inf
    g = np.random.default_rng(14)
    T = np.where(g.random(rows) < 0.1, 0.0, g.uniform(0.4, 1.5, rows))
    check(lib, dev, x, e, T)
    check(lib, dev, x, e, T, p=g.uniform(0.3, 1.0, rows))
    check(lib, dev, x, e, T, k=g.integers(0, 400, rows), floor=g.uniform(-0.02, 0.1, rows))
    if dtype == torch.float32:                                     # noise that takes many rounds
        order = torch.argsort(x[:, :], dim=1, descending=True, stable=True)
        rank = torch.empty_like(order).scatter_(1, order, torch.arange(vocab, device=dev).expand(rows, -1).contiguous())
        check(lib, dev, x, torch.exp(80 * (0.5 - (rank + 1) / vocab)).float(), T, k=g.integers(1, 3000, rows), p=g.uniform(0.2, 0.9, rows))


def test_masked_logits_of_the_processing(lib, cuda_device):
    """process_logits with a grammar's mask, then sampling: what is masked out is never drawn."""
    dev, rows, vocab = cuda_device, 6, 20000
    x, e = logits(15, rows, vocab, torch.float32, dev)
    allowed = torch.zeros(rows, vocab, dtype=torch.bool)
    for r, n in enumerate((1, 3, 40, 1000, 19999, 0)):
        allowed[r, torch.randperm(vocab, generator=torch.Generator("cpu").manual_seed(r))[:n]] = True
    words = np.packbits(allowed.numpy(), axis=1, bitorder="little").view(np.int32)
    kept = torch.empty(rows, vocab, device=dev)
    lib.process_logits(x, out=kept, allow_mask=torch.from_numpy(words.copy()).to(dev))
    for lim in (dict(), dict(k=50), dict(p=0.9), dict(floor=0.01)):
        got = check(lib, dev, kept, e, [0.9] * rows, **{n: [v] * rows for n, v in lim.items()})
        assert got[5] == -1 and all(bool(allowed[r, got[r]]) for r in range(5))
