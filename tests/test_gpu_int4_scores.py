"""paged_gqa_decode_int4 where scores are large or K lies at the ends of its range, in
each of the three ways that a call is split (a CTA for each sequence, clusters, shares)."""
import numpy as np
import pytest
import torch

from oracle import bf16 as OB, int4_kv as O4
from tests._util import bits
from tests.test_gpu_bs8 import rows, tables_for
from tests.test_gpu_int4 import check, close, decode, random_pages, rows_of, set_rows

pytestmark = pytest.mark.gpu
WAYS = ["own", "clusters", "shares"]


@pytest.fixture(scope="module")
def lib(cuda_device):
    from paged_kv_gqa_append_gb300 import build
    build.build()
    import paged_kv_gqa_append_gb300 as m
    return m


def case(way, seed):
    """Lengths and the bound that has them split this way."""
    if way == "own":
        lens = np.random.default_rng(seed).integers(33, 380, 100)
        lens[0] = 380
    else:
        lens = np.array([1500, 47, 333])
    pages = int(sum(-(-n // 16) for n in lens)) + 2
    return lens, pages, tables_for(seed + 1, lens, pages), 1 << 20 if way == "shares" else int(lens.max())


def times(pool, kv, by):
    for p in range(len(pool)):
        w = rows_of(pool, p, kv)
        set_rows(pool, p, kv, OB.from_f32_rne((OB.to_f64(w) * by).astype(np.float32)))


def same_key(pool, seed):
    """Every token's K row the same (one for each head)."""
    first = random_pages(seed, 1)
    for r in range(16):
        pool[:, :, O4.CODE_AT[0][r]] = first[:, :, O4.CODE_AT[0][0]]
        for i in range(4):
            pool[:, :, O4.SCALE_AT[0][r] + i] = first[:, :, O4.SCALE_AT[0][0] + i]


def equal_scores(lib, dev, way, size):
    """Tokens of the same key have the same score and probability, however large the score
    (here to 2^20 and beyond), so the output is the mean of the values: off by what the sums
    and products of the bound of test_gpu_int4.py are off by, without a term for scores."""
    lens, pages, bt, bound = case(way, 80)
    pool = random_pages(81, pages)
    same_key(pool, 82)
    q = rows(83, len(lens), 32, 64, scale=size)
    out, code = decode(lib, dev, q, pool, bt, lens, max_seq_len=bound)
    assert code == 0
    ref, span, reach, most = O4.attend(q, pool, bt, lens, 0.125)
    close(out, ref, span, 0 * reach, most, lens, way)


@pytest.mark.parametrize("size", [1.0, 2.0 ** 10, 2.0 ** 17])
def test_equal_scores_weigh_the_same(lib, cuda_device, size):
    equal_scores(lib, cuda_device, "own", size)


@pytest.mark.parametrize("size", [1.0, 2.0 ** 10, 2.0 ** 17])
@pytest.mark.parametrize("way", WAYS[1:])
def test_equal_scores_weigh_the_same_in_parts(lib, cuda_device, way, size):
    equal_scores(lib, cuda_device, way, size)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("way", WAYS)
def test_largest_keys(lib, cuda_device, way, sign):
    """K rows near 2^125 under ordinary queries: scores that 32 bits hold, so far apart that the
    best token has all the weight.  Heads whose best score is not beyond the error of the two
    are left out."""
    lens, pages, bt, bound = case(way, 84)
    pool = random_pages(85, pages)
    times(pool, 0, sign * 2.0 ** 121)
    if sign < 0:                                             # scales stay positive: minima above 0
        for p in range(pages):
            w = rows_of(pool, p, 0)
            w[..., 0] &= 0x7FFF
            set_rows(pool, p, 0, w)
    q = rows(86, len(lens), 32, 64)
    out, code = decode(lib, cuda_device, q, pool, bt, lens, max_seq_len=bound)
    assert code == 0
    got, seen = OB.to_f64(bits(out)), 0
    for s, n in enumerate(lens):
        v = O4.values(pool[bt[s, :-(-n // 16)]]).transpose(1, 2, 0, 3, 4).reshape(2, 8, -1, 64)[:, :, :n]
        x = 0.125 * np.einsum("ghd,gnd->ghn", OB.to_f64(q[s]).reshape(8, 4, 64), v[0])
        _, span, reach, _ = O4.attend(q[s:s + 1], pool, bt[s:s + 1], [n], 0.125)
        two = np.sort(x, -1)[..., -2:].reshape(32, 2)
        clear = two[:, 1] - two[:, 0] > 2.0 ** -14 * reach[0, :, 0] + 200
        want = np.take_along_axis(v[1][:, None], x.argmax(-1)[..., None, None], 2)[:, :, 0].reshape(32, 64)
        assert np.isfinite(got[s]).all()
        err = np.abs(got[s] - want) - 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -8) - 2.0 ** -18 * span[0]
        assert (err[clear] <= 0).all(), f"sequence {s}"
        seen += int(clear.sum())
    assert seen > 16 * len(lens)


@pytest.mark.parametrize("k,q", [(2.0 ** -112, 2.0 ** 111), (2.0 ** -60, 2.0 ** 60), (2.0 ** 118, 2.0 ** -118),
                                 (2.0 ** 40, 2.0 ** -40), (2.0 ** -30, 2.0 ** 80)])
@pytest.mark.parametrize("way", WAYS)
def test_small_keys_under_large_queries_and_the_reverse(lib, cuda_device, way, k, q):
    lens, pages, bt, bound = case(way, 87)
    pool = random_pages(88, pages)
    times(pool, 0, k)
    scale = 0.125 if k * q <= 1 else 0.125 / (k * q)
    check(lib, cuda_device, rows(89, len(lens), 32, 64, scale=q), pool, bt, lens, scale, max_seq_len=bound)


@pytest.mark.parametrize("way", WAYS)
def test_zero_queries_under_the_largest_keys(lib, cuda_device, way):
    """Every score is 0 then: the mean of the values."""
    lens, pages, bt, bound = case(way, 90)
    pool = random_pages(91, pages)
    times(pool, 0, 2.0 ** 121)
    q = rows(92, len(lens), 32, 64)
    q[:, ::2] = 0
    out, code = decode(lib, cuda_device, q, pool, bt, lens, max_seq_len=bound)
    assert code == 0
    ref, span, reach, most = O4.attend(q * 0, pool, bt, lens, 0.125)
    close(out[:, ::2], ref[:, ::2], span[:, ::2], 0 * reach[:, ::2], most[:, ::2], lens)


@pytest.mark.parametrize("score", [-1.6e38, -1.2e38, -9e37, 1.6e38])
@pytest.mark.parametrize("way", WAYS)
def test_equal_scores_at_the_ends_of_fp32(lib, cuda_device, way, score):
    """Keys of one value each, under which every token's score is this: the mean of the values."""
    lens, pages, bt, bound = case(way, 93)
    pool = random_pages(94, pages)
    for p in range(pages):
        w = rows_of(pool, p, 0)
        w[..., 0], w[..., 1] = 0, OB.from_f32_rne(np.float32(abs(score) / 64))
        set_rows(pool, p, 0, w)
    q = OB.from_f32_rne(np.full((len(lens), 32, 64), np.sign(score), np.float32))
    out, code = decode(lib, cuda_device, q, pool, bt, lens, scale=1.0, max_seq_len=bound)
    assert code == 0
    ref, span, reach, most = O4.attend(q * 0, pool, bt, lens, 1.0)
    close(out, ref, span, 0 * reach, most, lens)
